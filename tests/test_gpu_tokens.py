"""GPU parity of the token operators (HIP through the C ABI) against the
float64 oracle on the same inputs, at the sizes, strides and masks where
they can go wrong, and a run of them together.

Tolerances, from the arithmetic (a rounding is off by at most half a step:
2^-8 relative in bfloat16, 2^-24 in float32; a float32 sum is counted at a
whole step, 2^-23, an addition, as the matrix pipes' order and rounding
inside one instruction are their own):
 linear     a sum of K products goes through K/32 instructions and at most
            32 additions inside one: (K/32 + 32) 2^-23 sum |x w|; the
            activations have slopes up to 1.13 and are evaluated to
            2^-20 |z|; residual and output round once each.
 rope       the angle is right to 2^-25 of a turn and the cosine to 2 steps:
            4e-7; the norm's sum and quotient to 14 steps: 8e-7; together
            below 2^-19 (|u_p| + |u_q|) with the products' own rounding.
 attention  probabilities round to bfloat16 (2^-8 each, so 2^-8 of the
            weighted mean of |v|); scores (D <= 128: 4 instructions, 32
            additions) to 36 2^-23 sum |q k|, which exp passes on as a
            relative error, twice (sum and product); 1e-5 for the float32
            sums over up to 2^12 keys and the joins.
Outputs round to their type at the end.
"""
import numpy as np
import pytest
import torch

from oracle import tokens as ot

pytestmark = pytest.mark.gpu

BF, F32 = torch.bfloat16, torch.float32
STEP = {BF: 2.0 ** -8, F32: 2.0 ** -24}


@pytest.fixture(scope="module")
def gkd():
    import prompt_conditioned_keypoint_amd as m
    m.load()
    assert torch.cuda.is_available()
    return m


def randn(gen, *shape, dtype=BF, scale=1.0):
    return (torch.randn(*shape, generator=gen, device="cuda") * scale).to(dtype)


def rng(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    return g


def np64(t):
    return None if t is None else t.double().cpu().numpy()


def rounded(y, tol, dtype):
    return tol + STEP[dtype] * (np.abs(y) + tol)


# ------------------------------------------------------------------ linear
def linear_tol(y, size, K, dtype, residual):
    tol = 1.13 * (K / 32 + 32) * 2.0 ** -23 * size + 2.0 ** -20 * size
    if residual is not None:
        tol = tol + 2.0 ** -23 * (np.abs(y) + np.abs(residual))
    return rounded(y, tol, dtype)


def check_linear(gkd, M, K, N, act="none", bias=True, residual=True, out=BF, seed=0, **kw):
    print(f"[linear] M={M} K={K} N={N} {act} bias={bias} residual={residual} {out}", flush=True)
    g = rng(seed)
    x, w = randn(g, M, K), randn(g, N, K, scale=K ** -0.5)
    b = randn(g, N) if bias else None
    r = randn(g, M, N, dtype=out) if residual else None
    y = gkd.linear(x, w, bias=b, residual=r, act=act, out_dtype=out, **kw)
    assert y.dtype == out and y.shape == (M, N)
    want, size = ot.linear(np64(x), np64(w), np64(b), np64(r), act)
    err = np.abs(np64(y) - want)
    assert np.all(err <= linear_tol(want, size, K, out, np64(r))), err.max()


@pytest.mark.parametrize("act", ["none", "relu", "gelu", "quick_gelu", "silu"])
@pytest.mark.parametrize("out", [BF, F32])
def test_linear_activations(gkd, act, out):
    check_linear(gkd, 70, 192, 136, act, out=out)
    check_linear(gkd, 3, 192, 136, act, out=out, residual=False)


@pytest.mark.parametrize("M", [1, 2, 15, 16, 17, 33, 64, 65, 127, 129, 200, 257, 300])
@pytest.mark.parametrize("K,N", [(64, 16), (264, 257), (1000, 130), (8, 300)])
def test_linear_ragged_sizes(gkd, M, K, N):
    check_linear(gkd, M, K, N, seed=M)


@pytest.mark.parametrize("M,K,N", [(1, 1, 1), (5, 7, 3), (40, 33, 65), (130, 65, 129), (1, 1001, 40),
                                   (300, 517, 259)])
def test_linear_odd_widths_are_copied_first(gkd, M, K, N):
    check_linear(gkd, M, K, N, "silu", seed=K)
    check_linear(gkd, M, K, N, bias=False, residual=False, out=F32, seed=K)


@pytest.mark.parametrize("M,K,N", [(4200, 1024, 4096), (4097, 328, 4100), (1025, 4096, 1024),
                                   (19, 4096, 1030), (700, 2048, 320)])
def test_linear_large(gkd, M, K, N):
    check_linear(gkd, M, K, N, "gelu", seed=N)


@pytest.mark.parametrize("M,K,N,act,out,residual", [
    (5601, 520, 5797, "relu", BF, True),      # 256 x 256 tiles, two a workgroup, no even edge
    (5601, 250, 5800, "none", F32, True),
    (4000, 331, 4090, "silu", BF, False),     # one a workgroup, rows copied first
    (2100, 400, 1100, "gelu", F32, True),     # 128 x 128 tiles, a step or several
    (2100, 40, 1101, "none", BF, True),
    (1025, 72, 1023, "relu", F32, True),      # 128 x 64
    (20000, 24, 300, "none", BF, True),       # 128 x 128, two workgroups a CU
    (4130, 328, 4090, "none", F32, True),     # a whole round of 256 x 256 tiles and 34 rows apart
    (4470, 520, 4096, "gelu", BF, True),      # and 374 rows apart
])
def test_linear_tile_sizes(gkd, M, K, N, act, out, residual):
    check_linear(gkd, M, K, N, act, out=out, residual=residual, seed=K)


@pytest.mark.parametrize("M,N", [(3, 40), (64, 33), (150, 170), (1100, 1000), (2100, 1100), (4097, 4096),
                                 (20000, 300)])
@pytest.mark.parametrize("K", [72, 328])
def test_linear_reads_nothing_beside_its_rows(gkd, M, N, K):
    """NaN between the rows, before and behind them changes nothing."""
    g = rng(M + N)
    x, w, b = randn(g, M, K), randn(g, N, K), randn(g, N)
    want = gkd.linear(x, w, bias=b)

    def framed(t):
        buf = torch.full((t.shape[0] + 2, K + 24), float("nan"), dtype=BF, device="cuda")
        view = buf[1:-1, 8:8 + K]
        view.copy_(t)
        return view
    out = torch.full((M + 2, N + 3), 7.0, dtype=BF, device="cuda")
    got = gkd.linear(framed(x), framed(w), bias=b, out=out[1:-1, 1:-2])
    assert torch.equal(got, want)
    out[1:-1, 1:-2] = 7
    assert bool((out == 7).all())


@pytest.mark.parametrize("M,N", [(40, 600), (600, 600)])
def test_linear_rows_past_32_bit_offsets(gkd, M, N):
    """Rows 2^22 - 8 elements apart: the last of 600 lie past 2^31 elements."""
    g, K, ld = rng(6), 200, (1 << 22) - 8
    x, w, r = randn(g, M, K), randn(g, N, K), randn(g, M, N)
    want = gkd.linear(x, w, residual=r)

    def spread(t):
        far = torch.empty(t.shape[0], ld, dtype=BF, device="cuda")[:, :t.shape[1]]
        far.copy_(t)
        return far
    far = spread(r)
    assert torch.equal(gkd.linear(spread(x), spread(w), residual=far, out=far), want)


def test_linear_extreme_activations(gkd):
    """Activations far out: their limits, and NaN stays where it is."""
    x = torch.tensor([[200.0], [-200.0], [1e30], [-1e30], [0.0], [float("nan")]], device="cuda").to(BF)
    x = torch.nn.functional.pad(x, (0, 7))
    w = torch.nn.functional.pad(torch.ones(4, 1, device="cuda"), (0, 7)).to(BF)
    big = float(torch.tensor(1e30).to(BF))
    for act in ("relu", "gelu", "quick_gelu", "silu"):
        y = gkd.linear(x, w, act=act, out_dtype=F32).cpu()
        assert torch.equal(y[:5, 0], torch.tensor([200.0, 0.0, big, 0.0, 0.0])), (act, y)
        assert bool(torch.isnan(y[5]).all()), act


def test_linear_strided_rows_in_place_residual_and_untouched_padding(gkd):
    g = rng(3)
    M, K, N = 45, 72, 36
    xs, ws = randn(g, 3, 15, 2 * K), randn(g, N, K + 8)
    x, w = xs[:, :, K:], ws[:, :K]
    for out in (BF, F32):
        buf = torch.full((3, 15, N + 5), 7.0, dtype=out, device="cuda")
        y = buf[:, :, :N]
        y.copy_(randn(g, 3, 15, N))
        r = np64(y).reshape(M, N)
        got = gkd.linear(x, w, residual=y, out=y)
        assert got.data_ptr() == buf.data_ptr()
        want, size = ot.linear(np64(x).reshape(M, K), np64(w), None, r)
        assert np.all(np.abs(np64(y).reshape(M, N) - want) <= linear_tol(want, size, K, out, r))
        assert bool((buf[:, :, N:] == 7).all())
    # rows that start off 16-byte places: copied, same results
    xo = torch.empty(M, K + 1, dtype=BF, device="cuda")
    xo[:, :K] = x.reshape(M, K)
    a = gkd.linear(xo[:, :K], w)
    assert torch.equal(a, gkd.linear(x.reshape(M, K), w))


def test_linear_empty_and_refusals(gkd):
    w = torch.zeros(8, 16, dtype=BF, device="cuda")
    assert gkd.linear(torch.zeros(0, 16, dtype=BF, device="cuda"), w).shape == (0, 8)
    assert gkd.linear(torch.zeros(3, 16, dtype=BF, device="cuda"), w[:0]).shape == (3, 0)
    x = torch.zeros(4, 16, dtype=BF, device="cuda")
    with pytest.raises(gkd.GkdError) as e:
        gkd.linear(x[:1].expand(4, 16), w)
    assert e.value.status == 2
    with pytest.raises(gkd.GkdError) as e:
        gkd.linear(torch.zeros(65, dtype=BF, device="cuda")[1:].view(4, 16), w)
    assert e.value.status == 7
    with pytest.raises(gkd.GkdError) as e:
        gkd.linear(x[:, :15], w[:, :15], workspace=torch.empty(256, dtype=torch.uint8, device="cuda"))
    assert e.value.status == 4
    with pytest.raises(ValueError):
        gkd.linear(x, w, act="tanh")
    with pytest.raises(ValueError):
        gkd.linear(x, w, residual=torch.zeros(4, 8, dtype=F32, device="cuda"), out_dtype=BF)
    with pytest.raises(TypeError):
        gkd.linear(x.float(), w)


@pytest.mark.parametrize("act", ["relu", "gelu", "quick_gelu", "silu"])
@pytest.mark.parametrize("M", [40, 257])
def test_linear_activations_by_themselves(gkd, act, M):
    """Exact sums (one product each), so that the activation's own error is
    what there is: GELU to 2^-20 |z|, and relative to itself to 2^-12 in the
    tail down to -6; the quotients' exponent is rounded by 2^-22 of itself, its
    exponential, the sum, the reciprocal and the product by a step or two each."""
    x = torch.zeros(M, 8, dtype=BF, device="cuda")
    w = torch.zeros(300, 8, dtype=BF, device="cuda")
    x[:, 2] = torch.tensor(np.geomspace(1e-6, 4, M) * (-1.0) ** np.arange(M), device="cuda").to(BF)
    w[:, 2] = torch.linspace(1, 2, 300, device="cuda").to(BF)
    z = torch.outer(x[:, 2].double(), w[:, 2].double())
    got = gkd.linear(x, w, act=act, out_dtype=F32).double()
    if act == "relu":
        assert torch.equal(got, z.clamp(min=0))
        return
    if act == "gelu":
        want = z * torch.special.ndtr(z)
        err = (got - want).abs()
        assert bool((err <= 2.0 ** -20 * z.abs()).all()), (err / z.abs()).max()
        tail = (z < -1) & (z > -6)
        assert bool((err <= 2.0 ** -12 * want.abs())[tail].all()), (err / want.abs())[tail].max()
        return
    c = 1.702 if act == "quick_gelu" else 1.0
    gate = torch.sigmoid(c * z)
    want = z * gate
    tol = want.abs() * ((1 - gate) * (c * z.abs() * 2.0 ** -22 + 2.0 ** -23) + 2.0 ** -21)
    assert bool(((got - want).abs() <= tol).all()), ((got - want).abs() / want.abs()).max()


# -------------------------------------------------------------------- rope
def rope_inputs(g, B, T, Hq, Hk, D, rot, A, dtype, far=1000):
    rows = randn(g, B, T, (Hq + Hk) * D, dtype=dtype)
    q, k = rows[..., :Hq * D].unflatten(2, (Hq, D)), rows[..., Hq * D:].unflatten(2, (Hk, D))
    pos = (torch.rand(B, T, A, generator=g, device="cuda") * far).floor()
    freqs = torch.rand(A, rot // 2, generator=g, device="cuda")
    wq = randn(g, D, dtype=dtype)
    wk = randn(g, D, dtype=dtype)
    return q, k, pos, freqs, wq, wk


def check_rope(gkd, B, T, Hq, Hk, D, rot, A, dtype, norm, inter, seed=0, far=1000):
    print(f"[rope] {B}x{T} {Hq}/{Hk} heads of {D} rot {rot} axes {A} {dtype} norm={norm} inter={inter}",
          flush=True)
    q, k, pos, freqs, wq, wk = rope_inputs(rng(seed), B, T, Hq, Hk, D, rot, A, dtype, far)
    kw = dict(q_weight=wq, k_weight=wk) if norm else {}
    qo, ko = gkd.qk_norm_rope(q, k, pos, freqs, interleaved=inter, **kw)
    for x, y, w in ((q, qo, wq), (k, ko, wk)):
        want, size = ot.rope(np64(x), pos.cpu().numpy(), freqs.cpu().numpy(), np64(w) if norm else None,
                             1e-6, inter)
        err = np.abs(np64(y) - want)
        assert np.all(err <= rounded(want, 2.0 ** -19 * size, dtype)), err.max()


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("inter", [False, True])
@pytest.mark.parametrize("D,rot", [(64, 64), (128, 128), (64, 32), (96, 64), (80, 80), (80, 48), (256, 256),
                                   (512, 512), (40, 8), (24, 16)])
def test_rope_head_widths(gkd, dtype, inter, D, rot):
    check_rope(gkd, 2, 5, 3, 2, D, rot, 2, dtype, True, inter, seed=D)


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("D,rot", [(2, 2), (7, 4), (65, 62), (100, 6), (36, 20), (500, 500), (63, 2)])
def test_rope_any_width(gkd, dtype, D, rot):
    """Widths that are no whole 16-byte pieces, one by one."""
    check_rope(gkd, 2, 3, 2, 1, D, rot, 1, dtype, True, False, seed=D)
    check_rope(gkd, 1, 3, 1, 2, D, rot, 3, dtype, False, True, seed=D)


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("D,rot", [(64, 50), (96, 76), (128, 6), (256, 226), (512, 510), (80, 78), (40, 2)])
def test_rope_halves_of_no_whole_pieces(gkd, dtype, D, rot):
    """Split pairs whose halves end inside a 16-byte piece."""
    check_rope(gkd, 2, 37, 3, 2, D, rot, 2, dtype, True, False, seed=D)
    check_rope(gkd, 1, 5, 1, 1, D, rot, 1, dtype, False, False, seed=D)


@pytest.mark.parametrize("B,T,Hq,Hk,A", [(1, 1, 1, 1, 1), (1, 1, 32, 8, 1), (3, 129, 1, 1, 3), (2, 77, 5, 1, 8),
                                         (1, 700, 16, 16, 2)])
def test_rope_counts(gkd, B, T, Hq, Hk, A):
    check_rope(gkd, B, T, Hq, Hk, 64, 64, A, BF, True, False, seed=T)
    check_rope(gkd, B, T, Hq, Hk, 64, 64, A, BF, False, False, seed=T)


def test_rope_far_positions(gkd):
    """Positions of a million and more keep their angle (float32)."""
    check_rope(gkd, 1, 50, 2, 1, 64, 64, 1, F32, False, False, far=1 << 23)
    check_rope(gkd, 1, 50, 2, 1, 66, 64, 2, F32, False, False, far=1 << 23)


def test_rope_in_place_shared_table_queries_alone_and_strided_out(gkd):
    g = rng(5)
    q, k, pos, freqs, wq, wk = rope_inputs(g, 3, 9, 4, 2, 64, 64, 2, BF)
    pos = pos[0].contiguous()
    want = gkd.qk_norm_rope(q, k, pos.expand(3, 9, 2).contiguous(), freqs, wq, wk)
    alone, none = gkd.qk_norm_rope(q, None, pos, freqs, wq)
    assert none is None and torch.equal(alone, want[0])
    # a cache's slots, heads before tokens
    cache = torch.full((3, 2, 20, 64), 7.0, dtype=BF, device="cuda")
    view = cache.transpose(1, 2)[:, 4:13]
    got = gkd.qk_norm_rope(q, k, pos, freqs, wq, wk, k_out=view)
    assert torch.equal(got[0], want[0]) and torch.equal(view, want[1])
    assert bool((cache[:, :, :4] == 7).all()) and bool((cache[:, :, 13:] == 7).all())
    # off 16-byte places: the same values one by one
    off = torch.empty(3 * 9 * 4 * 64 + 1, dtype=BF, device="cuda")[1:].view(3, 9, 4, 64)
    off.copy_(q)
    o2, _ = gkd.qk_norm_rope(off, None, pos, freqs, wq)
    err = (o2.float() - want[0].float()).abs()
    assert bool((err <= 2 ** -7 * want[0].float().abs() + 1e-6).all())
    # in place, all kernels
    f2 = freqs[:, :21].contiguous()
    loose = gkd.qk_norm_rope(q, k, pos, f2, wq, wk)
    q2, k2 = q.clone(), k.clone()
    gkd.qk_norm_rope(q2, k2, pos, f2, wq, wk, q_out=q2, k_out=k2)
    assert torch.equal(q2, loose[0]) and torch.equal(k2, loose[1])
    gkd.qk_norm_rope(q, k, pos, freqs, wq, wk, q_out=q, k_out=k)
    assert torch.equal(q, want[0]) and torch.equal(k, want[1])
    gkd.qk_norm_rope(off, None, pos, freqs, wq, q_out=off)
    assert torch.equal(off, o2)


def test_rope_past_32_bit_offsets_and_two_streams(gkd):
    g = rng(15)
    for D, rot, inter in ((64, 64, False), (64, 42, False), (64, 42, True), (36, 20, False)):
        q, k, pos, freqs, wq, wk = rope_inputs(g, 2, 70, 3, 2, D, rot, 2, BF)
        want = gkd.qk_norm_rope(q, k, pos, freqs, wq, wk, interleaved=inter)
        far = torch.empty(2, 70, 1 << 25, dtype=BF, device="cuda")      # 2^25 elements a token: 9.4 GB
        fq, fk = far[:, :, :3 * D].unflatten(2, (3, D)), far[:, :, 1024:1024 + 2 * D].unflatten(2, (2, D))
        fq.copy_(q), fk.copy_(k)
        torch.cuda.synchronize()
        st = torch.cuda.Stream()
        with torch.cuda.stream(st):
            gkd.qk_norm_rope(fq, fk, pos, freqs, wq, wk, interleaved=inter, q_out=fq, k_out=fk)
        again = gkd.qk_norm_rope(q, k, pos, freqs, wq, wk, interleaved=inter)
        torch.cuda.synchronize()
        assert torch.equal(fq, want[0]) and torch.equal(fk, want[1])
        assert torch.equal(again[0], want[0]) and torch.equal(again[1], want[1])


def test_rope_zero_rows_and_refusals(gkd):
    z = torch.zeros(1, 2, 1, 64, dtype=BF, device="cuda")
    pos, freqs = torch.zeros(2, 1, device="cuda"), torch.ones(1, 32, device="cuda")
    w = torch.ones(64, dtype=BF, device="cuda")
    assert not bool(gkd.qk_norm_rope(z, None, pos, freqs, w)[0].any())     # eps keeps zero rows zero
    assert gkd.qk_norm_rope(z[:0], None, pos, freqs)[0].shape == (0, 2, 1, 64)
    with pytest.raises(gkd.GkdError) as e:
        gkd.qk_norm_rope(z, None, pos, torch.ones(1, 33, device="cuda"))
    assert e.value.status == 2
    with pytest.raises(ValueError):
        gkd.qk_norm_rope(z, None, pos[:1], freqs)
    with pytest.raises(ValueError):
        gkd.qk_norm_rope(z.transpose(1, 3), None, pos, freqs)
    with pytest.raises(TypeError):
        gkd.qk_norm_rope(z, z.float(), pos, freqs)
    with pytest.raises(TypeError):
        gkd.qk_norm_rope(z, None, pos.int(), freqs)


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("inter", [False, True])
@pytest.mark.parametrize("D,rot", [(64, 32), (64, 30), (96, 62), (80, 2), (40, 18), (128, 126), (65, 62)])
def test_rope_elements_past_rot_are_copied(gkd, dtype, inter, D, rot):
    """Infinities, NaN and zeros of both signs past rot come out as they are
    and stay out of their neighbours, whichever kernel runs."""
    print(f"[rope] D={D} rot={rot} {dtype} inter={inter}", flush=True)
    q, _, pos, freqs, wq, _ = rope_inputs(rng(D), 2, 9, 3, 1, D, rot, 2, dtype)
    q = q.contiguous()
    special = torch.tensor([float("inf"), 1.5, -float("inf"), -0.0, float("nan"), 2.5, 0.0, -3.0], device="cuda")
    q[..., rot:] = special.repeat(D // 8 + 1)[:D - rot].to(dtype)
    y, _ = gkd.qk_norm_rope(q, None, pos, freqs, interleaved=inter)
    rest, want = y[..., rot:].float(), q[..., rot:].float()
    assert torch.equal(rest.isnan(), want.isnan()) and torch.equal(rest.nan_to_num(9.0), want.nan_to_num(9.0))
    assert torch.equal(rest.signbit(), want.signbit())
    clean = q.clone()
    clean[..., rot:] = 0
    assert torch.equal(y[..., :rot], gkd.qk_norm_rope(clean, None, pos, freqs, interleaved=inter)[0][..., :rot])
    # an infinite square makes the norm infinite: finite elements become 0
    q[..., rot:] = 1
    q[..., -1] = float("inf")
    y, _ = gkd.qk_norm_rope(q, None, pos, freqs, wq, interleaved=inter)
    assert not bool(y[..., :-1].any()) and bool(y[..., -1].isnan().all())


@pytest.mark.parametrize("D,rot,inter", [(64, 64, False), (64, 64, True), (96, 76, False), (66, 62, True)])
def test_rope_float32_angles(gkd, D, rot, inter):
    """The pair (1, 0) comes out as (cos, sin): half a float32 step of 1
    (2^-25) for the rounding and 2^-30 for the angle and the functions."""
    q = torch.zeros(1, 3000, 1, D, device="cuda")
    i = torch.arange(rot // 2, device="cuda")
    p0, p1 = (2 * i, 2 * i + 1) if inter else (i, i + rot // 2)
    q[..., p0] = 1
    g = rng(D)
    pos = (torch.rand(3000, 2, generator=g, device="cuda") * 4000).floor()
    pos[:8, 0] = torch.arange(8, device="cuda")
    pos[:8, 1] = 0
    freqs = torch.rand(2, rot // 2, generator=g, device="cuda")
    freqs[0, :4] = torch.tensor([np.pi / 2, np.pi / 4, np.pi, 1e-4])
    y = gkd.qk_norm_rope(q, None, pos, freqs, interleaved=inter)[0].double()[0, :, 0]
    phi = (pos.double()[:, :, None] * freqs.double()).sum(1)
    err = max(float((y[:, p0] - phi.cos()).abs().max()), float((y[:, p1] - phi.sin()).abs().max()))
    assert err <= 2.0 ** -25 + 2.0 ** -30, err


# --------------------------------------------------------------- attention
def attn_inputs(g, B, Tq, Hq, Hk, D, P, S):
    q = randn(g, B, Tq, Hq, D)
    kv = randn(g, max(P, 1), 2, Hk, D)[:P]
    own = randn(g, B, max(S, 1), 2, Hk, D)[:, :S]
    return q, kv[:, 0], kv[:, 1], own[:, :, 0], own[:, :, 1]


def attn_tol(out, mean_abs, worst, D):
    delta = 36 * 2.0 ** -23 * worst + 1e-5
    return rounded(out, (2.0 ** -8 + 2 * delta) * mean_abs, BF)


def check_attn(gkd, B, Tq, Hq, Hk, D, P, S, own_len=None, q_len=None, mask=None, causal=False, scale=None,
               seed=0):
    print(f"[attn] B={B} Tq={Tq} {Hq}/{Hk} of {D} P={P} S={S} own_len={own_len} q_len={q_len} "
          f"mask={mask is not None} causal={causal}", flush=True)
    g = rng(seed)
    q, kp, vp, ko, vo = attn_inputs(g, B, Tq, Hq, Hk, D, P, S)
    dev = lambda v: None if v is None else torch.tensor(v, dtype=torch.int32, device="cuda")
    out = torch.full((B, Tq, Hq, D), 7.0, dtype=BF, device="cuda")
    got = gkd.prefix_attention(q, kp if P else None, vp if P else None, ko if S else None, vo if S else None,
                               own_len=dev(own_len), q_len=dev(q_len), own_mask=mask, causal=causal,
                               scale=scale, out=out)
    assert got.data_ptr() == out.data_ptr()
    want, mean_abs, worst = ot.prefix_attention(
        *(np64(t) for t in (q, kp, vp, ko, vo)), own_len, q_len, None if mask is None else mask.cpu().numpy(),
        causal, scale)
    y = np64(out)
    if q_len is not None:       # rows not asked for stay as they were
        for b, n in enumerate(q_len):
            assert (y[b, min(max(n, 0), Tq):] == 7).all()
            y[b, min(max(n, 0), Tq):] = 0
    err = np.abs(y - want)
    assert np.all(err <= attn_tol(want, mean_abs, worst, D)), err.max()


def masks(seed, B, S, p=0.6):
    return (torch.rand(B, S, generator=rng(seed), device="cuda") < p).to(torch.uint8)


@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("Hq,Hk", [(4, 4), (4, 2), (7, 1)])
@pytest.mark.parametrize("P,S", [(1, 1), (63, 65), (64, 64), (130, 0), (0, 130), (200, 31), (17, 257)])
@pytest.mark.parametrize("B,Tq", [(1, 1), (3, 1), (2, 5), (2, 70)])
def test_attention_shapes(gkd, D, Hq, Hk, P, S, B, Tq):
    check_attn(gkd, B, Tq, Hq, Hk, D, P, S, seed=P + S)


@pytest.mark.parametrize("D,Hq,Hk", [(64, 4, 2), (128, 6, 2)])
@pytest.mark.parametrize("Tq", [1, 3, 40, 90])
@pytest.mark.parametrize("causal", [False, True])
@pytest.mark.parametrize("P", [0, 150])
def test_attention_ragged_masked(gkd, D, Hq, Hk, Tq, causal, P):
    S = 140
    own_len = [140, Tq, 0, 77, 200, -3]
    q_len = [Tq, max(Tq - 2, 0), Tq, 1, Tq + 9, 0]
    check_attn(gkd, 6, Tq, Hq, Hk, D, P, S, own_len, q_len, masks(1, 6, S), causal, seed=Tq)
    check_attn(gkd, 6, Tq, Hq, Hk, D, P, S, own_len, None, None, causal, seed=Tq)


def test_attention_rows_without_keys_are_zero(gkd):
    m = torch.ones(3, 20, dtype=torch.uint8, device="cuda")
    m[1] = 0
    for Tq in (1, 2, 70):
        check_attn(gkd, 3, Tq, 4, 2, 64, 0, 20, [20, 20, 0], None, m)
        check_attn(gkd, 3, Tq, 4, 2, 64, 0, 20, [1, 0, 20], None, None, True)


@pytest.mark.parametrize("Tq", [1, 4, 70])
def test_attention_hidden_places_may_hold_anything(gkd, Tq):
    """NaN and infinities past own_len, under the mask and past q_len."""
    g = rng(11)
    B, Hq, Hk, D, P, S = 3, 4, 2, 128, 70, 100
    q, kp, vp, ko, vo = attn_inputs(g, B, Tq, Hq, Hk, D, P, S)
    own_len = torch.tensor([100, 33, 0], dtype=torch.int32, device="cuda")
    q_len = torch.tensor([Tq, max(1, Tq - 1), Tq], dtype=torch.int32, device="cuda")
    m = masks(2, B, S)
    kw = dict(own_len=own_len, q_len=q_len, own_mask=m)
    want = gkd.prefix_attention(q, kp, vp, ko, vo, out=torch.zeros_like(q), **kw)
    hidden = (m == 0) | (torch.arange(S, device="cuda") >= own_len[:, None])
    ko, vo, q = ko.clone(), vo.clone(), q.clone()
    ko[hidden], vo[hidden] = float("nan"), float("inf")
    vo[..., ::2][hidden] = float("nan")
    q[torch.arange(Tq, device="cuda") >= q_len[:, None]] = float("nan")
    got = gkd.prefix_attention(q, kp, vp, ko, vo, out=torch.zeros_like(q), **kw)
    assert torch.equal(got, want)


@pytest.mark.parametrize("B,Tq,Hq,Hk,D,P,S", [(5, 1, 8, 2, 128, 4000, 300), (2, 33, 4, 4, 64, 2304, 80),
                                              (1, 1, 16, 16, 64, 576, 80), (1, 2, 8, 1, 128, 9000, 64),
                                              (2, 260, 2, 1, 128, 700, 300)])
def test_attention_split_ranges(gkd, B, Tq, Hq, Hk, D, P, S):
    check_attn(gkd, B, Tq, Hq, Hk, D, P, S, [S - 7 * b for b in range(B)], None, None, True, seed=P)


# Batches whose rows are packed over the sequences for the prefix: few and
# many rows a sequence, more than 256 sequences, and one too many to pack.
PACKED = [(5, 1, 4, 2, 64, 1050, 70), (6, 3, 8, 2, 128, 1100, 150), (9, 16, 2, 2, 64, 1024, 33),
          (17, 33, 2, 2, 64, 2050, 40), (17, 20, 4, 1, 128, 2100, 130), (16, 97, 1, 1, 64, 3001, 97),
          (300, 1, 4, 2, 64, 1030, 33), (1024, 1, 2, 2, 64, 1024, 9), (1025, 1, 2, 2, 64, 1024, 9),
          (600, 18, 2, 2, 64, 2048, 20)]


@pytest.mark.parametrize("B,Tq,Hq,Hk,D,P,S", PACKED)
@pytest.mark.parametrize("causal", [False, True])
def test_attention_packed_rows(gkd, B, Tq, Hq, Hk, D, P, S, causal):
    some = [S, Tq, 0, S // 2 + 1, S + 60, -3, 1]
    less = [Tq, max(Tq - 2, 0), Tq, 1, Tq + 9, 0, Tq]
    own_len, q_len = [some[b % 7] for b in range(B)], [less[b % 7] for b in range(B)]
    check_attn(gkd, B, Tq, Hq, Hk, D, P, S, own_len, q_len, masks(1, B, S), causal, seed=P)
    if B < 100:
        check_attn(gkd, B, Tq, Hq, Hk, D, P, S, own_len, None, None, causal, seed=P)
        check_attn(gkd, B, Tq, Hq, Hk, D, P, S, None, [0] * B, None, causal, seed=P)
        check_attn(gkd, B, Tq, Hq, Hk, D, P, S, None, [0] * (B - 1) + [Tq], None, causal, seed=P)


@pytest.mark.parametrize("Tq", [1, 5, 40])
@pytest.mark.parametrize("D", [64, 128])
def test_attention_packed_rows_beside_hidden_places(gkd, Tq, D):
    """NaN and infinities past own_len, under the mask and past q_len, with
    strided caches and an output between other values."""
    g = rng(12)
    B, Hq, Hk, P, S = 18, 4, 2, 2100, 60
    q, kp, vp, ko, vo = attn_inputs(g, B, Tq, Hq, Hk, D, P, S)
    own_len = torch.tensor([60, 33, 0] * 6, dtype=torch.int32, device="cuda")
    q_len = torch.tensor([Tq, max(1, Tq - 1), 0, Tq, 1, Tq] * 3, dtype=torch.int32, device="cuda")
    m = masks(2, B, S)
    kw = dict(own_len=own_len, q_len=q_len, own_mask=m)
    want = gkd.prefix_attention(q, kp, vp, ko, vo, out=torch.full_like(q, 7.0), **kw)
    hidden = (m == 0) | (torch.arange(S, device="cuda") >= own_len[:, None])
    heads_first = lambda t: t.transpose(-2, -3).contiguous().transpose(-2, -3)
    ko, vo, kp, vp, q = (heads_first(t) for t in (ko, vo, kp, vp, q))
    ko[hidden], vo[hidden] = float("nan"), float("inf")
    vo[..., ::2][hidden] = float("nan")
    q[torch.arange(Tq, device="cuda") >= q_len[:, None]] = float("nan")
    buf = torch.full((B, Hq, Tq + 2, D + 8), 7.0, dtype=BF, device="cuda")
    out = buf[:, :, 1:-1, :D].transpose(1, 2)
    gkd.prefix_attention(q, kp, vp, ko, vo, out=out, **kw)
    assert torch.equal(out, want)
    out.fill_(7)
    assert bool((buf == 7).all())


def test_attention_shared_operands_and_no_keys(gkd):
    """One query row and one set of own keys for all sequences (strides of
    0), keys as values, and keys of no tokens."""
    g = rng(13)
    for P, Tq in ((70, 3), (1100, 3)):
        q, kp, vp, ko, vo = attn_inputs(g, 1, Tq, 4, 2, 64, P, 50)
        wide = [t.expand(6, *t.shape[1:]) for t in (q, ko, vo)]
        dense = [t.contiguous() for t in wide]
        assert torch.equal(gkd.prefix_attention(wide[0], kp, vp, wide[1], wide[2]),
                           gkd.prefix_attention(dense[0], kp, vp, dense[1], dense[2]))
        assert torch.equal(gkd.prefix_attention(dense[0], kp, kp, dense[1], dense[1]),
                           gkd.prefix_attention(dense[0], kp, kp.clone(), dense[1], dense[1].clone()))
        assert not bool(gkd.prefix_attention(q, kp[:0], vp[:0]).any())
        assert not bool(gkd.prefix_attention(q, kp[:0], vp[:0], ko[:, :0], vo[:, :0]).any())
        with pytest.raises(gkd.GkdError) as e:
            gkd.prefix_attention(wide[0], kp, vp, out=wide[0])
        assert e.value.status == 2


def test_attention_large_scores_and_scales(gkd):
    """Scores that jump by hundreds from chunk to chunk; a small and a large scale."""
    g = rng(9)
    q, kp, vp, ko, vo = attn_inputs(g, 2, 3, 4, 2, 64, 300, 100)
    kp = kp * torch.linspace(0.1, 12, 300, device="cuda").to(BF)[:, None, None]
    for scale in (1.0, 1e-6):
        got = np64(gkd.prefix_attention(q, kp, vp, ko, vo, scale=scale))
        want, mean_abs, worst = ot.prefix_attention(*(np64(t) for t in (q, kp, vp, ko, vo)), scale=scale)
        err = np.abs(got - want)
        assert np.all(err <= attn_tol(want, mean_abs, worst, 64)), err.max()


def test_attention_repeats_exactly_and_on_another_stream(gkd):
    g = rng(21)
    q, kp, vp, ko, vo = attn_inputs(g, 7, 1, 8, 2, 128, 3000, 200)
    a = gkd.prefix_attention(q, kp, vp, ko, vo)
    torch.cuda.synchronize()
    st = torch.cuda.Stream()
    with torch.cuda.stream(st):
        b = gkd.prefix_attention(q, kp, vp, ko, vo)
    st.synchronize()
    assert torch.equal(a, b)


def test_attention_long_cache_past_32_bit_offsets(gkd):
    """A token stride that puts the last keys more than 2^32 elements away."""
    S, stride = 300, 1 << 24         # 300 tokens, 2^24 elements apart: 10 GB of keys
    g = rng(2)
    ko = torch.zeros(S * stride, dtype=BF, device="cuda").view(1, S, stride)[:, :, :128].unflatten(2, (1, 128))
    src = randn(g, 1, S, 1, 128)
    ko.copy_(src)
    vo = randn(g, 1, S, 1, 128)
    for Tq in (1, 20):
        q = randn(g, 1, Tq, 2, 128)
        want = gkd.prefix_attention(q, None, None, src, vo)
        assert torch.equal(gkd.prefix_attention(q, None, None, ko, vo), want)
        want = gkd.prefix_attention(q, src[0], vo[0])
        assert torch.equal(gkd.prefix_attention(q, ko[0], vo[0]), want)


def test_attention_refusals(gkd):
    q = torch.zeros(2, 3, 4, 64, dtype=BF, device="cuda")
    kv = torch.zeros(5, 2, 64, dtype=BF, device="cuda")
    for bad in (dict(k_prefix=kv), dict(), dict(k_prefix=kv, v_prefix=kv[:4])):
        with pytest.raises(ValueError):
            gkd.prefix_attention(q, **bad)
    with pytest.raises(gkd.GkdError) as e:
        gkd.prefix_attention(q[:, :, :3], kv, kv)
    assert e.value.status == 5
    with pytest.raises(gkd.GkdError) as e:
        gkd.prefix_attention(q, kv, kv, scale=0.0)
    assert e.value.status == 4
    with pytest.raises(TypeError):
        gkd.prefix_attention(q, kv, kv, own_len=torch.zeros(2, dtype=torch.int64, device="cuda"))
    with pytest.raises(TypeError):
        gkd.prefix_attention(q.float(), kv, kv)


def one_hot_scores(B, Tq, Hq, Hk, D, P, S, dots):
    """Operands whose dot product with key j is `dots[j]` times a query row's
    sign (own keys behind the prefix's), exactly: one element of a head does it."""
    g = rng(P + S)
    q, kp, vp, ko, vo = (t.contiguous() for t in attn_inputs(g, B, Tq, Hq, Hk, D, P, S))
    for t in (q, kp, ko):
        t.zero_()
    q[..., 5] = 1
    q[:, 1::2, :, 5] = -1
    kp[..., 5] = dots[:P, None].to(BF)
    ko[..., 5] = dots[None, P:, None].to(BF)
    return q, kp, vp, ko, vo


@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("B,Tq,Hq,Hk,P,S", [
    (1, 2, 2, 1, 300, 70),        # thin tiles
    (1, 2, 1, 1, 9000, 64),       # and parts
    (2, 40, 2, 1, 300, 70),       # wide tiles
    (1, 130, 1, 1, 5000, 90),     # and parts
    (5, 2, 2, 1, 1100, 40),       # packed rows, thin tiles beside them
    (17, 20, 2, 1, 2100, 130)])   # packed rows, wide tiles beside them
@pytest.mark.parametrize("size", [1e5, 1e9, 1e10, 3.3e11, 1e20, 1e36])
def test_attention_scores_of_any_size(gkd, D, B, Tq, Hq, Hk, P, S, size):
    """Scores whose float32 steps are large numbers: the largest takes all."""
    print(f"[attn] B={B} Tq={Tq} {Hq}/{Hk} of {D} P={P} S={S} scores {size}", flush=True)
    j = torch.arange(P + S, device="cuda")
    dots = ((j * 7919) % (P + S) / (P + S) - 0.5) * size
    orders = {"mixed": dots, "rising": dots.sort()[0], "below zero": dots - size}
    for name, d in orders.items():
        # bfloat16 keeps 8 bits: one key above the rest and one below
        d = d.clone()
        top, low = (P + S // 2, 3) if name != "rising" else (P + S - 1, 0)
        d[top] = 2 * size if name != "below zero" else -0.25 * size
        d[low] = -3 * size
        q, kp, vp, ko, vo = one_hot_scores(B, Tq, Hq, Hk, D, P, S, d)
        got = gkd.prefix_attention(q, kp, vp, ko, vo, scale=1.0)
        v = torch.cat([vp.expand(B, -1, -1, -1), vo], 1)
        want = torch.empty_like(got)
        want[:, 0::2] = v[:, top, None].repeat_interleave(Hq // Hk, 2)
        want[:, 1::2] = v[:, low, None].repeat_interleave(Hq // Hk, 2)
        assert torch.equal(got, want), name


def test_attention_rows_with_huge_scores_leave_their_neighbours(gkd):
    """A row's bits are the same whatever the other rows of its wave see."""
    for D in (64, 128):
        for B, Tq, P, S in ((2, 60, 400, 90), (17, 20, 2100, 130)):
            q, kp, vp, ko, vo = attn_inputs(rng(31), B, Tq, 2, 1, D, P, S)
            want = gkd.prefix_attention(q, kp, vp, ko, vo)
            for size in (30.0, 1e8, 1e12):
                wild = q.clone()
                wild[:, ::3] *= size
                got = gkd.prefix_attention(wild, kp, vp, ko, vo)
                keep = torch.arange(Tq, device="cuda") % 3 != 0
                assert torch.equal(got[:, keep], want[:, keep]), (D, B, size)
                assert bool(got.isfinite().all()), (D, B, size)


@pytest.mark.parametrize("Tq", [1, 20])
@pytest.mark.parametrize("P,S,n", [((1 << 30) - 1, (1 << 30) - 1, (1 << 30) - 1),     # 2^31 - 2 keys
                                   ((1 << 30) - 1, (1 << 30) - 1, 1 << 29), ((1 << 30) - 64, (1 << 30) - 1, 70),
                                   (5, (1 << 30) - 1, (1 << 30) - 1)])
def test_attention_longest_lists_of_keys(gkd, Tq, P, S, n):
    """As many keys as the limits allow, one in memory (token strides of 0):
    equal scores, so the mean of the prefix's ones and the own keys' threes."""
    print(f"[attn] Tq={Tq} P={P} S={S} own_len={n}", flush=True)
    g = rng(4)
    q, k = randn(g, 1, Tq, 1, 64), randn(g, 1, 1, 64)
    one = torch.ones(1, 1, 64, dtype=BF, device="cuda")
    own_len = torch.tensor([n], dtype=torch.int32, device="cuda")
    got = gkd.prefix_attention(q, k.expand(P, 1, 64), one.expand(P, 1, 64), k[None].expand(1, S, 1, 64),
                               (3 * one)[None].expand(1, S, 1, 64), own_len=own_len)
    want = torch.tensor((P + 3 * n) / (P + n), device="cuda").to(BF)
    assert bool((got == want).all()), (got.float().min(), got.float().max(), want)


def test_sizes_past_32_bits_are_refused(gkd):
    """Sizes that a C int would cut to 5: views of little memory, and rows of
    one element (8 GB)."""
    n = 2 ** 32 + 5
    one = torch.ones(1, 1, 64, dtype=BF, device="cuda")
    q = torch.ones(1, 1, 1, 64, dtype=BF, device="cuda")
    out = torch.full_like(q, 7.0)
    for kw in (dict(k_prefix=one.expand(n, 1, 64), v_prefix=one.expand(n, 1, 64)),
               dict(k_own=one[None].expand(1, n, 1, 64), v_own=one[None].expand(1, n, 1, 64))):
        with pytest.raises(gkd.GkdError) as e:
            gkd.prefix_attention(q, out=out, **kw)
        assert e.value.status == 2
    with pytest.raises(gkd.GkdError) as e:
        gkd.qk_norm_rope(q.expand(1, 1, n, 64), None, torch.zeros(1, 1, device="cuda"),
                         torch.zeros(1, 32, device="cuda"), q_out=q.expand(1, 1, n, 64))
    assert e.value.status == 2 and "32 bits" in str(e.value)
    x = torch.empty(n, 1, dtype=BF, device="cuda")
    w = torch.ones(1, 1, dtype=BF, device="cuda")
    y = torch.empty(n, 1, dtype=BF, device="cuda")
    y[:8] = 7
    with pytest.raises(gkd.GkdError) as e:
        gkd.linear(x, w, out=y)
    assert e.value.status == 2 and bool((y[:8] == 7).all()) and bool((out == 7).all())


def test_attention_new_outputs_are_zero_past_q_len(gkd):
    """Without `out`, the rows of queries that are not computed are zeros."""
    for B, Tq, P in ((3, 5, 40), (17, 20, 2100)):
        q, kp, vp, ko, vo = attn_inputs(rng(41), B, Tq, 4, 2, 64, P, 30)
        q_len = torch.arange(B, dtype=torch.int32, device="cuda") % (Tq + 1)
        want = gkd.prefix_attention(q, kp, vp, ko, vo, q_len=q_len, out=torch.zeros_like(q))
        for _ in range(3):
            held = [torch.full_like(q, 7.0) for _ in range(4)]      # what new memory may hold
            torch.cuda.synchronize()
            del held
            assert torch.equal(gkd.prefix_attention(q, kp, vp, ko, vo, q_len=q_len), want)


@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("B,Tq,P,S", [(1, 1, 400, 0), (1, 1, 9000, 64), (3, 4, 0, 300), (2, 30, 300, 100),
                                      (5, 1, 1100, 40), (17, 20, 2100, 130)])
def test_attention_weights_add_to_one(gkd, D, B, Tq, P, S):
    """Where all probabilities but a few round down by almost half a step, the
    mean of ones is still 1: the sum takes what the product takes."""
    s = float(np.log(0.5 + 0.9 * 2.0 ** -9))
    hi = float(torch.tensor(s).to(BF))
    q, kp, vp, ko, vo = (t.contiguous() for t in attn_inputs(rng(1), B, Tq, 2, 1, D, P, S))
    for t in (q, kp, ko):
        t.zero_()
    q[..., :2] = 1
    for t in (kp, ko):
        t[..., 0], t[..., 1] = hi, s - hi
    kp[::32, :, :2] = 0         # every chunk of keys holds one that is not rounded
    ko[:, ::32, :, :2] = 0
    vp.fill_(1), vo.fill_(1)
    got = gkd.prefix_attention(q, kp, vp, ko, vo, scale=1.0)
    assert bool((got == 1).all()), got.float().min()


@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("B,Tq,P,S", [(2, 20, 300, 100), (2, 70, 700, 60), (17, 20, 2100, 130)])
@pytest.mark.parametrize("causal", [False, True])
def test_attention_growing_scores_in_wide_tiles(gkd, D, B, Tq, P, S, causal):
    """Scores that grow from chunk to chunk, so that the reference point moves
    by finite amounts while sums and outputs stand behind it."""
    q, kp, vp, ko, vo = attn_inputs(rng(9), B, Tq, 4, 2, D, P, S)
    q[:, ::4] *= 0.25                                   # rows that hardly move
    kp = kp * torch.linspace(0.1, 12, P, device="cuda").to(BF)[:, None, None]
    ko = ko * torch.linspace(12, 20, S, device="cuda").to(BF)[:, None, None]
    for scale in (1.0, 0.05, 1e-6):
        got = np64(gkd.prefix_attention(q, kp, vp, ko, vo, scale=scale, causal=causal))
        want, mean_abs, worst = ot.prefix_attention(*(np64(t) for t in (q, kp, vp, ko, vo)), causal=causal,
                                                    scale=scale)
        err = np.abs(got - want)
        assert np.all(err <= attn_tol(want, mean_abs, worst, D)), (scale, err.max())


@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("B,Tq,P,S", [(2, 40, 640, 64), (17, 20, 2112, 128), (1, 130, 5000, 64)])
@pytest.mark.parametrize("rise", [7.75, 8.0, 8.25, 0.5])
def test_attention_rises_about_the_slack(gkd, D, B, Tq, P, S, rise):
    """Scores (base 2) that rise by a little less or more than 8 from chunk to
    chunk, in some rows of a wave alone, and fall in others."""
    print(f"[attn] B={B} Tq={Tq} {D} P={P} S={S} rise {rise}", flush=True)
    q, kp, vp, ko, vo = (t.contiguous() for t in attn_inputs(rng(10), B, Tq, 2, 1, D, P, S))
    for t in (q, kp, ko):
        t[..., 1:] *= 0.125
    steps = (torch.arange(P + S, device="cuda") // 64 % 12) * rise
    kp[..., 0], ko[..., 0] = steps[:P, None].to(BF), steps[None, P:, None].to(BF)
    kinds = torch.tensor([1.0, 0.0, 0.5, -1.0, 1.0], device="cuda").to(BF)
    q[..., 0] = kinds[torch.arange(Tq, device="cuda") % 5][None, :, None]
    scale = float(np.log(2.0))
    got = gkd.prefix_attention(q, kp, vp, ko, vo, scale=scale)
    want, mean_abs, worst = ot.prefix_attention(*(np64(t) for t in (q, kp, vp, ko, vo)), scale=scale)
    err = np.abs(np64(got) - want)
    assert np.all(err <= attn_tol(want, mean_abs, worst, D)), err.max()
    # the rows that rise do not touch the bits of the others
    calm = q.clone()
    rising = torch.arange(Tq, device="cuda") % 5 == 0
    calm[:, rising, :, 0] = 0
    again = gkd.prefix_attention(calm, kp, vp, ko, vo, scale=scale)
    assert torch.equal(again[:, ~rising], got[:, ~rising])


# ------------------------------------------------------------ together
def test_a_block_over_image_tokens_and_prompt_rows(gkd):
    """A pre-projection block as a user builds it: image tokens give the
    shared keys, prompt sets attend to them and to their own rows, and a
    feed-forward pair follows, with a float32 residual stream; then the
    rows go to the heatmap call as kernels over the same tokens. Compared
    stage by stage with the oracle on the stage's own inputs."""
    B, R, C, H, W, Hq, Hk, D, F = 3, 12, 256, 6, 8, 4, 2, 64, 320
    g = rng(77)
    tokens = randn(g, 1, 5 + H * W, C)
    rows = randn(g, B, R, C)
    valid = masks(3, B, R, 0.7)
    wq, wkv = randn(g, Hq * D, C, scale=C ** -0.5), randn(g, 2 * Hk * D, C, scale=C ** -0.5)
    wo, w1, w2 = (randn(g, *s, scale=s[1] ** -0.5) for s in ((C, Hq * D), (F, C), (C, F)))
    bq, bkv, bo, b1, b2 = (randn(g, n, scale=0.1) for n in (Hq * D, 2 * Hk * D, C, F, C))
    gq, gk = (1 + 0.1 * randn(g, D, dtype=F32)).to(BF), (1 + 0.1 * randn(g, D, dtype=F32)).to(BF)
    # two axes; class and storage tokens and prompt rows have no place
    yx = torch.stack(torch.meshgrid(torch.arange(H), torch.arange(W), indexing="ij"), -1).reshape(-1, 2)
    pos = torch.cat([torch.zeros(5, 2), yx.float()]).cuda()
    base = 100.0 ** (-torch.arange(16) / 16)
    freqs = torch.zeros(2, 32)
    freqs[0, :16], freqs[1, 16:] = base, base
    freqs, none = freqs.cuda(), torch.zeros(R, 2, device="cuda")

    def run():
        kv = gkd.linear(tokens, wkv, bias=bkv).unflatten(2, (2, Hk, D))
        own = gkd.linear(rows, wkv, bias=bkv).unflatten(2, (2, Hk, D))
        q = gkd.linear(rows, wq, bias=bq).unflatten(2, (Hq, D))
        _, kp = gkd.qk_norm_rope(kv[:, :, 0], kv[:, :, 0], pos, freqs, None, gk)
        q, ko = gkd.qk_norm_rope(q, own[:, :, 0], none, freqs, gq, gk)
        o = gkd.prefix_attention(q, kp[0], kv[0, :, 1], ko, own[:, :, 1], own_mask=valid)
        x = gkd.linear(o.flatten(2), wo, bias=bo, residual=rows.float())
        h = gkd.linear(x.to(BF), w1, bias=b1, act="gelu")
        y = gkd.linear(h, w2, bias=b2, residual=x, out=torch.empty_like(x))
        return kv, own, q, kp, ko, o, x, h, y

    kv, own, q, kp, ko, o, x, h, y = run()
    heat, (idx, _, score) = gkd.kernel_heatmap(tokens.expand(B, -1, -1).contiguous(), kern_txt=y.to(BF),
                                               mask_txt=valid, token_hw=(H, W), token_skip=5)
    torch.cuda.synchronize()
    assert bool(torch.isfinite(score[valid > 0]).all()) and bool((idx[valid > 0] >= 0).all())

    def lin(got, xin, w, b, act="none", r=None):
        want, size = ot.linear(np64(xin).reshape(-1, xin.shape[-1]), np64(w), np64(b),
                               None if r is None else np64(r).reshape(-1, w.shape[0]), act)
        err = np.abs(np64(got).reshape(want.shape) - want)
        assert np.all(err <= linear_tol(want, size, w.shape[1], got.dtype,
                                        None if r is None else np64(r).reshape(want.shape)))
    lin(kv.flatten(2), tokens, wkv, bkv)
    lin(own.flatten(2), rows, wkv, bkv)
    want, size = ot.rope(np64(kv[:, :, 0]), pos[None].cpu().numpy(), freqs.cpu().numpy(), np64(gk))
    assert np.all(np.abs(np64(kp) - want) <= rounded(want, 2.0 ** -19 * size, BF))
    want, mean_abs, worst = ot.prefix_attention(np64(q), np64(kp[0]), np64(kv[0, :, 1]), np64(ko),
                                                np64(own[:, :, 1]), own_mask=valid.cpu().numpy())
    assert np.all(np.abs(np64(o) - want) <= attn_tol(want, mean_abs, worst, D))
    lin(x, o.flatten(2), wo, bo, r=rows)
    lin(h, x.to(BF), w1, b1, "gelu")
    lin(y, h, w2, b2, r=x)

    # the same run captured and replayed on new inputs, with eager work between
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        res = run()[-1]
    for seed in (1, 2, 3):
        tokens.copy_(randn(rng(seed), *tokens.shape))
        rows.copy_(randn(rng(seed + 50), *rows.shape))
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(res, run()[-1])


def test_two_captured_graphs_and_eager_calls_do_not_share_a_workspace(gkd):
    """Calls without a workspace argument get one each, in a graph too."""
    g = rng(8)
    sets = [attn_inputs(g, 6, 1, 8, 2, 64, 1500, 100) for _ in range(2)]
    want = [gkd.prefix_attention(*s) for s in sets]
    graphs, outs = [], []
    for s in sets:
        graphs.append(torch.cuda.CUDAGraph())
        with torch.cuda.graph(graphs[-1]):
            outs.append(gkd.prefix_attention(*s))
    streams = [torch.cuda.Stream() for _ in sets]
    torch.cuda.synchronize()
    for _ in range(4):
        for o in outs:
            o.zero_()
        torch.cuda.synchronize()
        for st, gr in zip(streams, graphs):
            with torch.cuda.stream(st):
                gr.replay()
        gkd.prefix_attention(*sets[0])
        torch.cuda.synchronize()
        for o, w in zip(outs, want):
            assert torch.equal(o, w)


def test_calls_from_several_threads_at_once(gkd):
    """Each thread's calls keep their own operands."""
    import threading
    sets = [attn_inputs(rng(60 + i), 4, 3, 4, 2, 64, 200 + 30 * i, 50) for i in range(4)]
    pos, freqs = torch.rand(3, 1, device="cuda"), torch.rand(1, 32, device="cuda")
    want = [(gkd.prefix_attention(*s), gkd.qk_norm_rope(s[0], s[3][:, :3], pos, freqs)) for s in sets]
    torch.cuda.synchronize()
    bad = []

    def work(i):
        with torch.cuda.stream(torch.cuda.Stream()):
            for _ in range(50):
                got = gkd.prefix_attention(*sets[i]), gkd.qk_norm_rope(sets[i][0], sets[i][3][:, :3], pos, freqs)
                torch.cuda.current_stream().synchronize()
                if not (torch.equal(got[0], want[i][0]) and torch.equal(got[1][0], want[i][1][0])
                        and torch.equal(got[1][1], want[i][1][1])):
                    bad.append(i)
    threads = [threading.Thread(target=work, args=(i,)) for i in range(4)]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    assert not bad
