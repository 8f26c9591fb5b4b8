"""The projections on an MI355X, through the binding, against plain 64-bit
forms of their definitions.

Most inputs are small whole numbers (times powers of two), so that every
product and every partial sum is exact in fp32 whatever its order (their sums
stay under 2^24 units): an fp32 result then has to be the exact one, bit for
bit, and a 16-bit result its rounding to nearest even.  Inputs that are not
exact are compared within bounds that the test derives."""
import pytest
import torch

pytestmark = pytest.mark.gpu

BF, HF, F4 = torch.bfloat16, torch.float16, torch.float32


@pytest.fixture(scope="module")
def p():
    from hyper_connection_residual_amd import projections
    assert torch.cuda.is_available()
    return projections


def case(*what):
    print("case:", *what, flush=True)


def whole(gen, shape, most, dtype, unit=1.0):
    return (torch.randint(-most, most + 1, shape, generator=gen, device="cuda") * unit).to(dtype)


def new_gen(seed):
    gen = torch.Generator(device="cuda")
    gen.manual_seed(seed)
    return gen


def exact(got, want64):
    """got is the correctly rounded want64 (whose values fp32 holds)."""
    assert torch.equal(want64.float().double(), want64)
    assert torch.equal(got, want64.float().to(got.dtype))


def plain_project(x, W, adapter=None, A=None, B=None, scale=None):
    y = x.double() @ W.double().T
    if adapter is not None:
        for a in range(A.shape[0]):
            mine = adapter == a
            s = 1.0 if scale is None else scale[a].double()
            y[mine] += s * ((x[mine].double() @ A[a].double().T) @ B[a].double().T)
    return y


def project_inputs(T, K, N, dtype, rank, adapters, seed=0):
    """|x| <= 3, |W| <= 3: W's sums stay under 9 K; |A|, |B| <= 1, each sparse: v under 3 K / 8, its sums
    under 3 K r / 64 / 8; scale 1, 2 or 4."""
    gen = new_gen(seed)
    x, W = whole(gen, (T, K), 3, dtype), whole(gen, (N, K), 3, dtype)
    if not adapters:
        return x, W, None, None, None, None
    A = whole(gen, (adapters, rank, K), 1, dtype) * (torch.rand((adapters, rank, K), generator=gen, device="cuda") < 0.125)
    B = whole(gen, (adapters, N, rank), 1, dtype) * (torch.rand((adapters, N, rank), generator=gen, device="cuda") < 0.125)
    scale = 2.0 ** torch.randint(0, 3, (adapters,), generator=gen, device="cuda").float()
    adapter = torch.randint(-1, adapters + 1, (T,), generator=gen, device="cuda", dtype=torch.int32)  # -1 and n: none
    return x, W, adapter, A, B, scale


@pytest.mark.parametrize("out_dtype", [None, F4], ids=["same", "fp32"])
@pytest.mark.parametrize("dtype", [BF, HF], ids=["bf16", "fp16"])
@pytest.mark.parametrize("T,K,N,rank,adapters", [
    (1, 2560, 2560, 16, 8), (1, 8, 1, 8, 1), (1, 72, 17, 24, 2), (1, 1000, 4100, 40, 3), (1, 2568, 250, 64, 5), (1, 264, 5000, 72, 2),
    (1, 640, 300, 128, 4), (2, 64, 3, 8, 2), (3, 72, 16, 24, 3), (15, 136, 17, 32, 4),
    (16, 2560, 130, 64, 5), (17, 520, 127, 128, 3), (25, 2560, 320, 32, 6), (33, 1000, 257, 16, 7), (64, 2560, 66, 8, 40),
    (65, 64, 128, 16, 4), (65, 8, 5, 8, 2), (130, 2568, 127, 40, 9), (200, 10240, 320, 64, 16), (333, 2560, 1000, 128, 16),
    (700, 640, 129, 16, 1), (1025, 200, 640, 8, 3), (1, 2560, 2560, 0, 0), (40, 264, 100, 0, 0), (515, 1288, 383, 0, 0),
    (2048, 2560, 2560, 16, 2),
    (1, 264, 5000, 16, 2), (1, 264, 5000, 24, 3), (12, 136, 5000, 16, 4), (7, 136, 5001, 24, 4), (30, 264, 8192, 8, 9),
    # tiles of 64 and 128 tokens, with and without splits of K
    (40, 2560, 10240, 16, 9), (100, 264, 9001, 8, 5), (129, 2568, 4109, 0, 0), (200, 2560, 4109, 24, 3), (300, 520, 4100, 128, 20),
    (333, 2560, 3001, 0, 0), (333, 10240, 2560, 64, 16), (700, 640, 4229, 16, 1), (1025, 200, 6400, 48, 7), (2000, 328, 2049, 16, 3),
    (600, 10240, 700, 40, 4), (1100, 2560, 1290, 8, 2), (130, 10240, 2570, 0, 0), (36, 2080, 9080, 8, 6),
    (45, 8720, 4215, 0, 0), (45, 8720, 4215, 16, 4), (129, 2568, 4109, 16, 4), (333, 10240, 2560, 0, 0),
    # tiles of 256 x 256 with splits of K, and in whole rounds with the rest by itself
    (2479, 3816, 1843, 0, 0), (1801, 2528, 2429, 16, 5), (1232, 3056, 3237, 0, 0), (810, 4080, 3163, 24, 4), (2096, 7912, 941, 0, 0),
    (2786, 8208, 399, 8, 3), (6600, 2568, 2560, 0, 0), (6600, 2568, 2560, 16, 6), (8193, 264, 10240, 8, 4),
    # tiles of 256 x 256: odd and even steps, a last step in part, ranks of one and of more chunks, few and many adapters
    (3001, 200, 4099, 0, 0), (3001, 128, 4099, 16, 2), (2900, 72, 4200, 8, 1), (2817, 1000, 4609, 48, 5), (4097, 320, 2900, 128, 30),
])
def test_project_is_exact_on_whole_numbers(p, T, K, N, rank, adapters, dtype, out_dtype):
    case("project", T, K, N, rank, adapters, dtype, out_dtype)
    x, W, adapter, A, B, scale = project_inputs(T, K, N, dtype, rank, adapters)
    y = p.project(x, W, adapter, A, B, scale, out_dtype=out_dtype)
    assert y.dtype == (out_dtype or dtype)
    want = plain_project(x, W, adapter, A, B, scale)
    assert float(want.abs().max()) < 2 ** 16  # (fp16 holds it)
    exact(y, want)


@pytest.mark.parametrize("T,N", [(1, 200), (5, 200), (40, 200), (300, 200), (300, 4100), (2000, 2049), (50000, 200)])
def test_project_one_adapter_for_all_and_one_per_token(p, T, N):
    case("project adapters", T, N)
    x, W, adapter, A, B, _ = project_inputs(T, 320, N, BF, 16, 7)
    for ad in (torch.full_like(adapter, 0), torch.full_like(adapter, 3), torch.full_like(adapter, 6), torch.full_like(adapter, 7), torch.arange(T, device="cuda", dtype=torch.int32) % 7, torch.full_like(adapter, -1),
               torch.full_like(adapter, 1 << 30), torch.full_like(adapter, -(1 << 31))):
        exact(p.project(x, W, ad, A, B, out_dtype=F4), plain_project(x, W, ad, A, B))


@pytest.mark.parametrize("T,N", [(1, 640), (20, 640), (90, 640), (400, 4000), (1500, 1500), (17000, 640)])
@pytest.mark.parametrize("dtype", [BF, HF], ids=["bf16", "fp16"])
def test_project_random_within_its_bound(p, T, N, dtype):
    """Random inputs in fp32 out.  A sum of n fp32 terms, in any order and with each addition off by at most a unit
    in its last place (2^-23: the matrix cores need not round to nearest), is off by at most n 2^-23 times the
    sum of the terms' magnitudes.  v: K terms of |A||x| (K 2^-23); y: K + r terms and v's error."""
    case("project random", T, N, dtype)
    K, n, r = 2560, 5, 40
    gen = new_gen(T)
    x = torch.randn((T, K), generator=gen, device="cuda").to(dtype)
    W, A, B = (0.02 * torch.randn(s, generator=gen, device="cuda").to(dtype) for s in ((N, K), (n, r, K), (n, N, r)))
    scale = torch.rand((n,), generator=gen, device="cuda") + 0.5
    adapter = torch.randint(-1, n, (T,), generator=gen, device="cuda", dtype=torch.int32)
    y = p.project(x, W, adapter, A, B, scale, out_dtype=F4).double()
    size = plain_project(x.abs(), W.abs(), adapter, A.abs(), B.abs(), scale)
    assert bool(((y - plain_project(x, W, adapter, A, B, scale)).abs() <= (2 * K + 2 * r + 8) * 2.0 ** -23 * size).all())
    # fp32 outputs of one small sum are far nearer than that: the mean error is that of some tens of roundings
    rel = float((y - plain_project(x, W, adapter, A, B, scale)).norm() / y.norm())
    print("relative error", rel, flush=True)
    assert rel < 64 * 2.0 ** -24
    y16 = p.project(x, W, adapter, A, B, scale)
    assert torch.equal(y16, y.float().to(dtype))  # the same sums, rounded once


@pytest.mark.parametrize("T,N,K", [(1, 61, 136), (4, 61, 136), (50, 61, 136), (400, 5003, 136), (50000, 61, 136), (1801, 2429, 2528),
                                   (6600, 2561, 2568)])
def test_project_strided_rows_and_untouched_neighbours(p, T, N, K):
    case("project strided", T, N, K)
    x, W, adapter, A, B, scale = project_inputs(T, K, N, BF, 8, 3)
    wide = torch.full((T, K + 64), float("nan"), dtype=BF, device="cuda")
    wide[:, 16:K + 16] = x
    for pitch, dtype in ((N + 3, BF), (N + 6, BF), (N + 3, F4), (N + 4, F4)):
        out = torch.full((T + 2, pitch), 7.0, dtype=dtype, device="cuda")
        got = p.project(wide[:, 16:K + 16], W, adapter, A, B, scale, out=out[1:-1, 1:N + 1])
        assert got.data_ptr() == out[1:-1, 1:N + 1].data_ptr()
        exact(got, plain_project(x, W, adapter, A, B, scale))
        assert bool((out[0] == 7).all()) and bool((out[-1] == 7).all()) and bool((out[:, 0] == 7).all())
        assert bool((out[:, N + 1:] == 7).all())


@pytest.mark.parametrize("dtype", [BF, HF], ids=["bf16", "fp16"])
@pytest.mark.parametrize("T,N,K", [(8, 150, 200), (48, 150, 200), (200, 150, 200), (300, 4100, 200), (333, 2560, 10240), (2000, 2049, 200),
                                   (1801, 2429, 2528), (6600, 2560, 2568),
                                   (50000, 150, 200)])
def test_project_tokens_see_only_their_own_row_and_adapter(p, T, N, K, dtype):
    """Infinities and NaN in one token's row or one adapter's weights stay in the tokens that use them."""
    case("project isolation", T, N, K, dtype)
    x, W, adapter, A, B, scale = project_inputs(T, K, N, dtype, 24, 4)
    adapter = (torch.arange(T, device="cuda", dtype=torch.int32) % 5) - 1
    want = p.project(x, W, adapter, A, B, scale)
    A2, B2, s2, x2 = A.clone(), B.clone(), scale.clone(), x.clone()
    A2[1], B2[2], s2[3] = float("nan"), float("inf"), float("nan")
    x2[T // 2] = float("nan")
    got = p.project(x2, W, adapter, A2, B2, s2)
    clean = (adapter == -1) | (adapter == 0)
    clean[T // 2] = False
    assert torch.equal(got[clean], want[clean])
    assert bool(torch.isnan(got[adapter == 1]).all()) and bool(torch.isnan(got[adapter == 3]).all())
    assert not bool(torch.isfinite(got[adapter == 2]).any()) and bool(torch.isnan(got[T // 2]).all())


@pytest.mark.parametrize("T,N", [(1, 150), (8, 150), (48, 150), (300, 4100), (2000, 2049), (50000, 150)])
def test_project_subnormal_weights(p, T, N):
    """fp16 weights of all 11 bits below the normal numbers, times whole numbers: exact in fp32."""
    case("project subnormal", T, N)
    x, W, adapter, A, B, _ = project_inputs(T, 200, N, HF, 24, 4)
    gen = new_gen(T)
    B = (torch.randint(-1023, 1024, B.shape, generator=gen, device="cuda") * 2.0 ** -24).to(HF)
    x, A = whole(gen, x.shape, 1, HF), whole(gen, A.shape, 1, HF)  # (sums of 24 x 200 x 1023 < 2^24)
    W = (torch.randint(-1023, 1024, W.shape, generator=gen, device="cuda") * 2.0 ** -24).to(HF)
    exact(p.project(x, W, out_dtype=F4), plain_project(x, W))  # (sums of 200 x 1023)
    W.zero_()
    exact(p.project(x, W, adapter, A, B, out_dtype=F4), plain_project(x, W, adapter, A, B))


@pytest.mark.parametrize("dtype", [BF, HF], ids=["bf16", "fp16"])
@pytest.mark.parametrize("T,N", [(1, 150), (8, 150), (48, 150), (300, 4100), (2000, 2049), (50000, 150)])
def test_project_infinite_inputs_stay_infinities(p, T, N, dtype):
    """All weights above zero, so that one infinite input makes every sum of its token infinite, and no NaN."""
    case("project infinite", T, N, dtype)
    x, W, adapter, A, B, scale = project_inputs(T, 200, N, dtype, 24, 4)
    W, A, B, scale = W.abs() + 1, A.abs() + 1, B.abs() + 1, scale.abs() + 1
    adapter = torch.arange(T, device="cuda", dtype=torch.int32) % 5
    want = p.project(x, W, adapter, A, B, scale, out_dtype=F4)
    x2 = x.clone()
    x2[T // 2, 77] = float("inf")
    got = p.project(x2, W, adapter, A, B, scale, out_dtype=F4)
    assert bool((got[T // 2] == float("inf")).all())
    got[T // 2] = want[T // 2]
    assert torch.equal(got, want)


def plain_experts(x, W, offsets, rows, gate, R):
    y = torch.zeros((R, W.shape[1] // (2 if gate else 1)), dtype=torch.float64, device="cuda")
    at = offsets.tolist()
    for e in range(W.shape[0]):
        lo, hi = min(max(at[e], 0), R), min(max(at[e + 1], 0), R)
        if lo < hi:
            i = torch.arange(lo, hi, device="cuda") if rows is None else rows[lo:hi].long()
            ok = (i >= 0) & (i < x.shape[0])
            xe = x.double()[i.clamp(0, x.shape[0] - 1)] * ok[:, None]
            h = xe @ W[e].double().T
            if gate:
                g, u = h.chunk(2, dim=1)
                h = g / (1 + torch.exp(-g)) * u
            y[lo:hi] = h
    return y


def groups(gen, R, E, kind):
    """Offsets of E groups of R rows: even, some empty, one that has all, or the last rows in no group."""
    if kind == "one":
        at = torch.zeros(E + 1, dtype=torch.int64)
        at[E // 2 + 1:] = R
    else:
        cuts = torch.randint(0, R + 1, (E - 1,), generator=torch.Generator().manual_seed(R + E)).sort().values
        at = torch.cat([torch.zeros(1, dtype=torch.int64), cuts, torch.tensor([R])])
        if kind == "short":
            at = at.clamp(max=R - max(1, R // 4))
    return at.int().cuda()


@pytest.mark.parametrize("gate", [False, True], ids=["plain", "gate"])
@pytest.mark.parametrize("R,K,N,E,kind,gather", [
    (1, 2560, 64, 1, "even", False), (1, 8, 1, 3, "one", True), (8, 2560, 257, 64, "even", True),
    (37, 136, 16, 64, "even", False), (64, 1024, 130, 64, "short", True), (200, 72, 33, 70, "even", True),
    (300, 264, 48, 20, "short", False), (500, 64, 129, 3, "one", True), (777, 520, 65, 9, "even", True),
    (1806, 256, 127, 32, "short", True), (4100, 128, 96, 5, "even", False), (3000, 2560, 256, 130, "even", True),
    (6000, 1288, 200, 4, "even", True),
    (40, 136, 70, 4, "even", False), (600, 72, 300, 70, "even", True), (1146, 2280, 58, 1, "one", False),
    # tiles of 64 and 128 rows, rings of two and three stages
    (900, 520, 2000, 10, "even", True), (1300, 1000, 1400, 20, "short", False), (1300, 200, 2800, 20, "even", True),
    (500, 64, 3000, 3, "one", True), (4100, 128, 1500, 5, "even", False), (700, 2560, 2560, 20, "even", True),
    (1833, 72, 1892, 40, "even", True),
    # tiles of 256 x 256
    (3794, 72, 1692, 29, "short", True), (20011, 136, 700, 5, "even", True), (20011, 264, 700, 100, "short", True), (12000, 2560, 1100, 9, "even", False),
    (9000, 72, 3001, 2, "one", True),
])
@pytest.mark.parametrize("dtype", [BF, HF], ids=["bf16", "fp16"])
def test_expert_project(p, R, K, N, E, kind, gather, gate, dtype):
    """Plain: exact on whole numbers.  Gated: the products g and u are exact (units of 2^-6, so that silu is not
    saturated), and silu(g) u in fp32 is off by: the exponential (its argument's rounding, |g| log2(e) 2^-24 of the
    result, and 2 units of v_exp's), an addition, a division (2.5 units), a product: under (|g| + 8) 2^-22; then the rounding
    of the output, half of eps, and 2^-25 (half the last place of fp16's subnormals)."""
    case("experts", R, K, N, E, kind, gather, gate, dtype)
    gen = new_gen(R + K)
    X = max(1, R // 3) if gather else R
    x = whole(gen, (X, K), 3, dtype)
    W = whole(gen, (E, 2 * N if gate else N, K), 3, dtype, 2.0 ** -6 if gate else 1.0)
    offsets = groups(gen, R, E, kind)
    rows = torch.randint(-1, X + 1, (R,), generator=gen, device="cuda", dtype=torch.int32) if gather else None
    for out_dtype in (dtype, F4):
        out = torch.full((R, N), 5.0, dtype=out_dtype, device="cuda")
        y = p.expert_project(x, W, offsets, rows=rows, gate=gate, out=out)
        end = int(offsets[-1])
        assert bool((y[end:] == 5).all())  # rows of no group
        want = plain_experts(x, W, offsets, rows, gate, R)[:end]
        if not gate:
            exact(y[:end], want)
        else:
            g = plain_experts(x, W[:, :N].contiguous(), offsets, rows, False, R)[:end]
            half = torch.finfo(out_dtype).eps / 2
            bound = want.abs() * ((g.abs() + 8) * 2.0 ** -22 + half) + (2.0 ** -25 if out_dtype == HF else 2.0 ** -126)
            off = (y[:end].double() - want).abs()
            assert bool((off <= bound).all()), float((off / bound).max())


def test_expert_offsets_out_of_order_stay_inside(p):
    """Offsets below 0 and above R are clamped to [0, R]; a row outside x is zeros."""
    case("expert offsets")
    gen = new_gen(3)
    x, W = whole(gen, (40, 64), 3, BF), whole(gen, (3, 32, 64), 3, BF)
    offsets = torch.tensor([-5, 10, 30, 1000], dtype=torch.int32, device="cuda")
    rows = torch.arange(40, dtype=torch.int32, device="cuda")
    rows[7], rows[20] = 40, -(1 << 31)
    y = p.expert_project(x, W, offsets, rows=rows, out_dtype=F4)
    exact(y, plain_experts(x, W, offsets, rows, False, 40))
    assert bool((y[7] == 0).all()) and bool((y[20] == 0).all())


def test_expert_offsets_out_of_order_with_more_tiles_than_32_bits_count(p):
    case("offsets out of order, many")
    gen = new_gen(5)
    R, E, N = 2800000, 112000, 128
    offsets = torch.zeros(E + 1, dtype=torch.int32, device="cuda")
    offsets[1::2] = R  # every other group claims all rows
    x, W = whole(gen, (R, 8), 3, BF), whole(gen, (1, N, 8), 3, BF)
    out = torch.full((R + 2, N), 777, dtype=BF, device="cuda")
    before, after = out[0].clone(), out[-1].clone()
    p.expert_project(x, W.expand(E, N, 8).contiguous(), offsets, out=out[1:-1])
    want = p.project(x, W[0])  # (up to 72: whole numbers)
    assert torch.equal(out[0], before) and torch.equal(out[-1], after)
    assert bool(((out[1:-1] == want) | (out[1:-1] == before)).all())


@pytest.mark.parametrize("R,N", [(10, 150), (600, 150), (600, 3000), (50000, 150)])
def test_experts_see_only_their_own_rows_and_weights(p, R, N):
    case("expert isolation", R, N)
    gen = new_gen(R)
    x, W = whole(gen, (R, 200), 3, BF), whole(gen, (5, N, 200), 3, BF)
    offsets = torch.tensor([0, R // 5, R // 5, R // 2, R - 1, R], dtype=torch.int32, device="cuda")
    want = p.expert_project(x, W, offsets)
    W2, x2 = W.clone(), x.clone()
    W2[1], W2[2], x2[0] = float("nan"), float("nan"), float("inf")
    got = p.expert_project(x2, W2, offsets)
    keep = torch.ones(R, dtype=torch.bool, device="cuda")
    keep[R // 5:R // 2] = False
    assert bool(torch.isnan(got[~keep]).all())
    keep[0] = False
    assert torch.equal(got[keep], want[keep])


@pytest.mark.parametrize("R", [9, 400, 50000])
def test_expert_project_strided(p, R):
    case("experts strided", R)
    gen = new_gen(R)
    x, W = whole(gen, (R, 72), 3, HF), whole(gen, (3, 45, 72), 3, HF)
    offsets = torch.tensor([0, R // 3, R // 3 + 1, R], dtype=torch.int32, device="cuda")
    wide = torch.full((R, 96), float("inf"), dtype=HF, device="cuda")
    wide[:, 8:80] = x
    out = torch.full((R, 51), 7.0, dtype=F4, device="cuda")
    exact(p.expert_project(wide[:, 8:80], W, offsets, out=out[:, 3:48]), plain_experts(x, W, offsets, None, False, R))
    assert bool((out[:, :3] == 7).all()) and bool((out[:, 48:] == 7).all())


def plain_route(logits, k, renorm):
    """From the definition, on the CPU, in 64 bits."""
    z = logits.cpu().double()
    z = torch.where(torch.isnan(z), -torch.inf, z).clamp(max=3.4028234663852886e38)
    T, E = z.shape
    top, ids = (t[:, :k] for t in z.sort(dim=1, descending=True, stable=True))
    some = top > -torch.inf
    peak = torch.where(some[:, :1], top[:, :1], 0.0)
    e = torch.exp(top - peak)
    total = e.sum(1, keepdim=True) if renorm else torch.exp(z - peak).sum(1, keepdim=True)
    w = torch.where(some, e / total, 0.0)
    ids = torch.where(some, ids, -1)
    slots = [(int(ids[t, s]), t, s) for t in range(T) for s in range(k) if ids[t, s] >= 0]
    slots.sort(key=lambda x: x[0])  # (stable: tokens stay in order)
    rows, pos = torch.full((T * k,), -1), torch.full((T, k), -1)
    counts = torch.zeros(E + 1, dtype=torch.int64)
    for i, (e_, t, s) in enumerate(slots):
        rows[i], pos[t, s] = t, i
        counts[e_ + 1] += 1
    return ids, w, counts.cumsum(0), rows, pos


def check_route(p, logits, k, renorm):
    ids, w, offsets, rows, pos = p.route(logits, k, renorm=renorm)
    want = plain_route(logits, k, renorm)
    for got, right in zip((ids, offsets, rows, pos), (want[0], want[2], want[3], want[4])):
        assert torch.equal(got.cpu().long(), right)
    # exp's argument is rounded (|z| 2^-24, at most 104 before exp is 0) and exp, its sum of up to E terms and the division are off by
    # some units each: under (104 + E + 8) 2^-23 of the weight; 2^-126 where it underflows
    off = (w.cpu().double() - want[1]).abs()
    assert bool((off <= want[1] * (logits.shape[1] + 112) * 2.0 ** -23 + 2.0 ** -126).all()), float(off.max())


@pytest.mark.parametrize("renorm", [True, False])
@pytest.mark.parametrize("T,E,k,dtype", [
    (1, 1, 1, F4), (1, 64, 8, F4), (3, 2, 2, BF), (8, 64, 8, F4), (17, 63, 6, HF), (16, 65, 1, F4), (33, 128, 4, BF),
    (100, 129, 32, F4), (400, 200, 20, F4), (300, 100, 17, BF), (128, 512, 8, F4), (129, 60, 8, F4), (300, 257, 7, BF), (1000, 8, 8, F4), (2049, 128, 8, F4),
    (5000, 512, 2, HF), (64, 200, 3, F4), (65, 200, 3, F4), (128, 96, 16, HF), (4097, 64, 8, BF), (8200, 256, 17, F4), (33000, 40, 2, F4), (60, 300, 5, F4),
])
def test_route(p, T, E, k, dtype, renorm):
    case("route", T, E, k, dtype, renorm)
    gen = new_gen(T + E)
    z = 3 * torch.randn((T, E), generator=gen, device="cuda")
    z[torch.rand((T, E), generator=gen, device="cuda") < 0.05] = float("-inf")
    z[torch.rand((T,), generator=gen, device="cuda") < 0.1] = float("-inf")  # padding
    check_route(p, z.to(dtype), k, renorm)


@pytest.mark.parametrize("T", [9, 500])
def test_route_ties_masks_and_extremes(p, T):
    case("route extremes", T)
    gen = new_gen(T)
    z = torch.randint(-2, 3, (T, 70), generator=gen, device="cuda").float()  # many ties
    z[:, 5] *= -0.0  # (zeros of both signs are equal)
    z[0] = float("nan")
    z[1] = float("-inf")
    z[2, 3:] = float("-inf")  # fewer than k are left
    z[3, 7], z[3, 9] = float("inf"), float("inf")
    z[4] = -3.0e38
    z[5, 11] = 3.0e38
    z[6, ::2] = float("nan")
    z[7] = 1e-40
    z[8] = -104.0
    z[8, 0] = 0.0
    for renorm in (True, False):
        check_route(p, z, 8, renorm)


def test_route_strided_logits(p):
    case("route strided")
    z = torch.randn((50, 100), generator=new_gen(1), device="cuda")
    a, b = p.route(z[:, 3:67], 4), p.route(z[:, 3:67].contiguous(), 4)
    assert all(torch.equal(x, y) for x, y in zip(a, b))


def test_route_many_tokens(p):
    """More tokens than the blocks' least size allows for (their tokens grow), against torch on the GPU."""
    case("route many")
    T, E, k = 100003, 40, 3
    z = torch.randn((T, E), generator=new_gen(2), device="cuda")
    ids, w, offsets, rows, pos = p.route(z, k)
    want = z.sort(dim=1, descending=True, stable=True).indices[:, :k]
    assert torch.equal(ids.long(), want)
    flat, order = want.flatten().sort(stable=True)
    assert torch.equal(rows.long(), order // k)
    assert torch.equal(pos.flatten().long()[order], torch.arange(T * k, device="cuda"))
    assert torch.equal(offsets.long(), torch.searchsorted(flat, torch.arange(E + 1, device="cuda")))


@pytest.mark.parametrize("out_dtype", [BF, HF, F4], ids=["bf16", "fp16", "fp32"])
@pytest.mark.parametrize("dtype", [BF, HF, F4], ids=["bf16", "fp16", "fp32"])
@pytest.mark.parametrize("T,k,C", [(1, 1, 1), (1, 8, 2560), (5, 3, 127), (40, 8, 264), (300, 2, 1000), (70, 32, 72)])
def test_combine_is_exact_on_whole_numbers(p, T, k, C, dtype, out_dtype):
    case("combine", T, k, C, dtype, out_dtype)
    gen = new_gen(T + C)
    rows = T * k + 3
    y = whole(gen, (rows, C), 15, dtype)
    pos = torch.randint(-2, rows + 2, (T, k), generator=gen, device="cuda", dtype=torch.int32)
    w = torch.randint(0, 9, (T, k), generator=gen, device="cuda") / 4.0
    ok = (pos >= 0) & (pos < rows)
    want = (y.double()[pos.clamp(0, rows - 1).long()] * torch.where(ok, w, 0.0).double()[:, :, None]).sum(1)
    w[~ok] = float("nan")  # (a position outside y adds nothing)
    exact(p.expert_combine(y, pos, w, out_dtype=out_dtype), want)
    wide = torch.full((rows, C + 9), float("nan"), dtype=dtype, device="cuda")
    wide[:, 8:C + 8] = y
    out = torch.full((T, C + 5), 7.0, dtype=out_dtype, device="cuda")
    exact(p.expert_combine(wide[:, 8:C + 8], pos, w, out=out[:, 4:C + 4]), want)
    assert bool((out[:, :4] == 7).all()) and bool((out[:, C + 4:] == 7).all())


def test_nothing_to_do(p):
    case("empty")
    x, W = torch.zeros((0, 64), dtype=BF, device="cuda"), torch.zeros((2, 32, 64), dtype=BF, device="cuda")
    assert p.project(x, W[0]).shape == (0, 32)
    assert p.expert_project(x, W, torch.zeros(3, dtype=torch.int32, device="cuda")).shape == (0, 32)
    ids, w, offsets, rows, pos = p.route(torch.zeros((0, 8), device="cuda"), 2)
    assert ids.shape == (0, 2) and offsets.tolist() == [0] * 9 and rows.numel() == 0
    none = torch.zeros((4, 0), dtype=torch.int32, device="cuda")
    assert bool((p.expert_combine(W[0], none, none.float()) == 0).all())
    one = torch.ones((3, 64), dtype=BF, device="cuda")
    A, B = torch.zeros((0, 8, 64), dtype=BF, device="cuda"), torch.zeros((0, 32, 8), dtype=BF, device="cuda")
    none = torch.zeros(3, dtype=torch.int32, device="cuda")
    assert torch.equal(p.project(one, W[1], none, A, B), p.project(one, W[1]))


def test_offsets_past_32_bits(p):
    """Weights, tokens and outputs that lie more than 4 GiB into their tensors."""
    case("past 32 bits")
    gen = new_gen(5)
    E, N, K = 70, 4096, 8192  # 4.7 GB of weights
    W = torch.zeros((E, N, K), dtype=BF, device="cuda")
    W[-1, -40:] = whole(gen, (40, K), 3, BF)
    x = whole(gen, (5, K), 3, BF)
    for R in (5, 2000):
        rows = (torch.arange(R, device="cuda") % 5).int()
        offsets = torch.zeros(E + 1, dtype=torch.int32, device="cuda")
        offsets[-1] = R
        y = p.expert_project(x, W, offsets, rows=rows, out_dtype=F4)
        exact(y[:, -40:], (x.double() @ W[-1, -40:].double().T)[rows.long()])
        assert bool((y[:, :-40] == 0).all())
    del W, y
    T = 300000  # 4.9 GB of tokens
    x = torch.zeros((T, K), dtype=BF, device="cuda")
    x[-3:] = whole(gen, (3, K), 3, BF)
    W = whole(gen, (9, K), 3, BF)
    y = p.project(x, W)
    exact(y[-3:], x[-3:].double() @ W.double().T)
    assert bool((y[:-3] == 0).all())
    rows = torch.tensor([T - 1, 0, T - 2], dtype=torch.int32, device="cuda")
    y = p.expert_project(x, W[None], torch.tensor([0, 3], dtype=torch.int32, device="cuda"), rows=rows, out_dtype=F4)
    exact(y, x[rows.long()].double() @ W.double().T)
    del x, y
    C, R = 4096, 600000  # 4.9 GB of rows
    y = torch.zeros((R, C), dtype=BF, device="cuda")
    y[-1] = whole(gen, (C,), 3, BF)
    pos = torch.tensor([[R - 1, 0]], dtype=torch.int32, device="cuda")
    exact(p.expert_combine(y, pos, torch.tensor([[2.0, 1.0]], device="cuda"), out_dtype=F4)[0], 2 * y[-1].double())


def layer(p, x, w, k):
    """The second read's way through the router and the experts."""
    logits = p.project(x, w["router"], out_dtype=F4)
    ids, weights, offsets, rows, pos = p.route(logits, k)
    h = p.expert_project(x, w["up"], offsets, rows=rows, gate=True)
    y = p.expert_project(h, w["down"], offsets, out_dtype=F4)
    return p.expert_combine(y, pos, weights, out_dtype=F4), (logits, ids, weights, offsets, rows, pos, h, y)


@pytest.mark.parametrize("T", [1, 8, 40, 600])
def test_read_project_route_experts_together(p, T):
    """As a layer runs them: the read's image through an adapted projection, then through router, experts and combine,
    and the result as the next read's pending write.  Every stage against its definition on the stage before, within
    the sums' bound (n terms: n 2^-23 of their magnitudes) and its rounding."""
    from hyper_connection_residual_amd import binding, workloads as wl
    case("together", T)
    inp = wl.config_inputs(2, T=T)
    dev = lambda a: torch.from_numpy(a).cuda()  # noqa: E731
    R, w_norm = dev(inp.R), dev(inp.w_norm)
    Wd, Wu = dev(inp.W_down.view("int16")), dev(inp.W_up.view("int16"))
    _, x, _ = binding.read(R, w_norm, Wd, Wu, pending=dev(inp.pending))
    gen = new_gen(T)
    rand = lambda *s: (0.02 * torch.randn(s, generator=gen, device="cuda")).to(BF)  # noqa: E731
    E, k, F, K, n, r = 16, 4, 320, 2560, 3, 16
    adapter = (torch.arange(T, device="cuda") % 4 - 1).int()
    W, A, B = rand(1280, K), rand(n, r, K), rand(n, 1280, r)
    q = p.project(x, W, adapter, A, B)
    size = plain_project(x.abs(), W.abs(), adapter, A.abs(), B.abs())
    want = plain_project(x, W, adapter, A, B)
    assert bool(((q.double() - want).abs() <= (2 * K + 2 * r + 8) * 2.0 ** -23 * size + 2.0 ** -8 * want.abs()).all())

    w = {"router": rand(E, K), "up": rand(E, 2 * F, K), "down": rand(E, K, F)}
    out, (logits, ids, weights, offsets, rows, pos, h, y) = layer(p, x, w, k)
    want = x.double() @ w["router"].double().T
    assert bool(((logits.double() - want).abs() <= K * 2.0 ** -23 * (x.abs().double() @ w["router"].abs().double().T)).all())
    right = plain_route(logits, k, True)
    assert all(torch.equal(a.cpu().long(), b) for a, b in zip((ids, offsets, rows, pos), (right[0], right[2], right[3], right[4])))
    R_ = T * k
    gu = plain_experts(x, w["up"], offsets, rows, False, R_)
    d = K * 2.0 ** -23 * plain_experts(x.abs(), w["up"].abs(), offsets, rows, False, R_)
    g, u, dg, du = gu[:, :F], gu[:, F:], d[:, :F], d[:, F:]
    silu = g / (1 + torch.exp(-g))
    # |silu'| <= 1.1
    bound = 1.1 * dg * (u.abs() + du) + silu.abs() * du + (silu * u).abs() * ((g.abs() + 8) * 2.0 ** -22 + 2.0 ** -8)
    assert bool(((h.double() - silu * u).abs() <= bound).all())
    want = plain_experts(h, w["down"], offsets, None, False, R_)
    size = plain_experts(h.abs(), w["down"].abs(), offsets, None, False, R_)
    assert bool(((y.double() - want).abs() <= F * 2.0 ** -23 * size).all())
    terms = y.double()[pos.long()] * weights.double()[:, :, None]
    assert bool(((out.double() - terms.sum(1)).abs() <= (k + 1) * 2.0 ** -23 * terms.abs().sum(1)).all())
    pending = out[:, None, :].expand(T, 4, 2560).contiguous()
    mixed, _, _ = binding.read(R, w_norm, Wd, Wu, pending=pending)
    assert bool(torch.isfinite(mixed).all())


@pytest.mark.parametrize("T", [2, 70, 300])
def test_captured_and_replayed(p, T):
    """The chain in a graph, replayed with other inputs and eager work between; every replay equals the eager result bit for bit."""
    case("graph", T)
    gen = new_gen(T)
    rand = lambda *s: (0.05 * torch.randn(s, generator=gen, device="cuda")).to(BF)  # noqa: E731
    K, E, F, k = 256, 12, 64, 3
    w = {"router": rand(E, K), "up": rand(E, 2 * F, K), "down": rand(E, K, F)}
    W, A, B = rand(512, K), rand(4, 16, K), rand(4, 512, 16)
    adapter = (torch.arange(T, device="cuda") % 5 - 1).int()
    x = torch.randn((T, K), generator=gen, device="cuda").to(BF)

    def step():
        return p.project(x, W, adapter, A, B), layer(p, x, w, k)[0]

    step()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        held = step()
    for turn in range(4):
        x.copy_(torch.randn((T, K), generator=gen, device="cuda"))
        adapter.copy_(torch.randint(-1, 4, (T,), generator=gen, device="cuda"))
        graph.replay()
        torch.cuda.synchronize()
        got = [t.clone() for t in held]
        want = step()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(got, want)), turn


def test_two_graphs_and_two_streams_at_once(p):
    """Two captured projections replayed together on two streams, and eager calls on a third: no scratch is shared."""
    case("two graphs")
    ins = [project_inputs(40, 2560, 512, BF, 16, 4, seed=s) for s in range(2)]
    big = project_inputs(300, 2560, 512, BF, 16, 4, seed=9)
    want = [plain_project(*i) for i in ins] + [plain_project(*big)]
    p.project(*big)
    graphs, outs, streams = [], [], [torch.cuda.Stream() for _ in range(3)]
    torch.cuda.synchronize()
    for i in ins:
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            outs.append(p.project(*i))
        graphs.append(g)
    torch.cuda.synchronize()
    for _ in range(20):
        for g, s in zip(graphs, streams):
            with torch.cuda.stream(s):
                g.replay()
        got = p.project(*big, stream=streams[2])
    torch.cuda.synchronize()
    for y, right in zip(outs + [got], want):
        exact(y, right)


def test_stream_argument(p):
    """A torch stream or a raw handle; the work runs there, after what the stream already holds."""
    case("stream")
    x, W, adapter, A, B, scale = project_inputs(30, 512, 256, HF, 16, 4)
    want = plain_project(x, W, adapter, A, B, scale)
    logits = torch.randn((200, 32), generator=new_gen(1), device="cuda")
    y, pos, w = whole(new_gen(2), (60, 64), 3, BF), torch.arange(60, device="cuda").int().view(30, 2), torch.ones((30, 2), device="cuda")
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    for stream in (s, s.cuda_stream, torch.cuda.current_stream(), 0):
        got = p.project(x, W, adapter, A, B, scale, stream=stream)
        ids = p.route(logits, 3, stream=stream)[0]
        z = p.expert_combine(y, pos, w, stream=stream)
        e = p.expert_project(x, W[None], torch.tensor([0, 30], dtype=torch.int32, device="cuda"), stream=stream)
        torch.cuda.synchronize()
        exact(got, want)
        assert torch.equal(ids.long(), logits.topk(3).indices)
        exact(z, y.double().view(30, 2, 64).sum(1))
        exact(e, plain_project(x, W))


def test_same_bits_every_time(p):
    """No atomics: results do not depend on the order in which workgroups run."""
    case("repeat")
    gen = new_gen(8)
    for T, N in ((7, 700), (100, 700), (400, 4000), (3000, 4200)):
        x = torch.randn((T, 2560), generator=gen, device="cuda").to(BF)
        W = torch.randn((N, 2560), generator=gen, device="cuda").to(BF)
        A, B = torch.randn((3, 16, 2560), generator=gen, device="cuda").to(BF), torch.randn((3, N, 16), generator=gen, device="cuda").to(BF)
        adapter = (torch.arange(T, device="cuda") % 3).int()
        one = p.project(x, W, adapter, A, B, out_dtype=F4)
        for _ in range(5):
            assert torch.equal(p.project(x, W, adapter, A, B, out_dtype=F4), one)


def same(got, want):
    """Equal, NaN to NaN."""
    return bool(((got == want) | (torch.isnan(got) & torch.isnan(want))).all())


SIZES_OF_ALL_KERNELS = [(1, 150, 200), (8, 150, 200), (48, 150, 200), (300, 4100, 200), (2000, 2049, 200), (50000, 150, 200),
                        # A x in splits, tiles and wide tiles with splits of K, and in two parts
                        (20, 150, 10240), (333, 2560, 10240), (1801, 2429, 2528), (6600, 2560, 2568)]


@pytest.mark.parametrize("dtype", [BF, HF], ids=["bf16", "fp16"])
@pytest.mark.parametrize("T,N,K", SIZES_OF_ALL_KERNELS)
def test_project_infinite_inputs_meet_infinite_and_smallest_weights(p, T, N, K, dtype):
    """One token's v is infinite at every rank, and one rank of B holds infinities, or the smallest numbers of its type.
    The signs of an output's weights agree, so that every term of the token's sums is an infinity of that sign."""
    case("project infinite, twice", T, N, K, dtype)
    x, W, adapter, A, B, scale = project_inputs(T, K, N, dtype, 24, 4)
    sign = (1 - 2 * (torch.arange(N, device="cuda") % 2)).to(dtype)
    W, A, B = (W.abs() + 1) * sign[:, None], A.abs() + 1, (B.abs() + 1) * sign[None, :, None]
    adapter = torch.arange(T, device="cuda", dtype=torch.int32) % 5
    adapter[T // 2] = 2
    x2 = x.clone()
    x2[T // 2, 77] = float("inf")
    least = torch.finfo(dtype).smallest_normal * torch.finfo(dtype).eps
    for value in (float("inf"), least, 7 * least):
        B2 = B.clone()
        B2[2, :, 5] = (value * sign.double()).to(dtype)
        assert bool((B2[2, :, 5] != 0).all())
        want = p.project(x, W, adapter, A, B2, scale, out_dtype=F4)
        got = p.project(x2, W, adapter, A, B2, scale, out_dtype=F4)
        assert torch.equal(got[T // 2], sign.float() * float("inf")), value
        got[T // 2] = want[T // 2]
        assert same(got, want)
        if value == float("inf"):
            assert same(want.double(), plain_project(x, W, adapter, A, B2, scale))


@pytest.mark.parametrize("dtype", [BF, HF], ids=["bf16", "fp16"])
@pytest.mark.parametrize("T,N,K", SIZES_OF_ALL_KERNELS)
def test_project_infinite_scale(p, T, N, K, dtype):
    """scale times the sum over the ranks: an infinity of the sum's sign, NaN where the sum is zero."""
    case("project infinite scale", T, N, K, dtype)
    x, W, adapter, A, B, scale = project_inputs(T, K, N, dtype, 24, 4)
    adapter = (torch.arange(T, device="cuda", dtype=torch.int32) + 1) % 5
    scale[1], scale[3] = float("inf"), float("-inf")
    got = p.project(x, W, adapter, A, B, scale, out_dtype=F4)
    assert same(got.double(), plain_project(x, W, adapter, A, B, scale))

    # with an infinite input as well, and weights above zero: infinities of the scale's sign, but for those of W x
    W, A, B, x2 = W.abs() + 1, A.abs() + 1, B.abs() + 1, x.clone()
    adapter[T // 2] = 1
    x2[T // 2, 77] = float("inf")
    B[1, :, 5] = float("inf")
    got = p.project(x2, W, adapter, A, B, scale, out_dtype=F4)
    assert bool((got[T // 2] == float("inf")).all())
    got[T // 2] = 0.0
    want = plain_project(x, W, adapter, A, B, scale)
    want[T // 2] = 0.0
    assert same(got.double(), want)


@pytest.mark.parametrize("E,k", [(64, 8), (128, 16), (200, 20), (512, 32)])
@pytest.mark.parametrize("T", [5, 64, 300, 5000])
def test_route_every_token_the_same_experts(p, T, E, k):
    """A wave's tokens then count at the same places, turn after turn: the token's number is its rank."""
    case("route same", T, E, k)
    z = torch.randn((1, E), generator=new_gen(T + E), device="cuda").expand(T, E).contiguous()
    ids, w, offsets, rows, pos = p.route(z, k)
    best = z[0].topk(k).indices
    assert torch.equal(ids.long(), best.expand(T, k))
    place = torch.empty_like(best)
    place[best.argsort()] = torch.arange(k, device="cuda")
    t = torch.arange(T, device="cuda")
    assert torch.equal(pos.long(), place[None] * T + t[:, None])
    assert torch.equal(rows.long(), t.repeat(k))
    assert int(offsets[-1]) == T * k


def test_single_columns_of_any_stride(p):
    case("single columns")
    gen = new_gen(4)
    x, W = whole(gen, (30, 64), 3, BF), whole(gen, (1, 64), 3, BF)
    buffer = torch.full((400,), 7.0, dtype=F4, device="cuda")
    out = buffer.as_strided((30, 1), (6, 3), 5)
    exact(p.project(x, W, out=out), plain_project(x, W))
    pos = torch.arange(29, -1, -1, device="cuda").int().view(30, 1)
    w = torch.full((30, 1), 2.0, device="cuda")
    exact(p.expert_combine(out, pos, w), 2 * plain_project(x, W).flip(0))
    ids, weights, offsets, rows, _ = p.route(out, 1)
    assert bool((ids == 0).all()) and bool((weights == 1).all()) and offsets.tolist() == [0, 30]
    assert torch.equal(rows.long(), torch.arange(30, device="cuda"))
    buffer.as_strided((30, 1), (6, 3), 5).fill_(7.0)
    assert bool((buffer == 7).all())


@pytest.mark.parametrize("raw", [False, True], ids=["stream", "handle"])
def test_stream_argument_waits_for_what_the_stream_holds(p, raw):
    """The inputs get their values on the given stream, behind work that is still running when the calls are made."""
    case("stream order", raw)
    gen = new_gen(7)
    s = torch.cuda.Stream()
    stream = s.cuda_stream if raw else s
    x0, W, adapter, A, B, scale = project_inputs(30, 512, 256, HF, 16, 4)
    x1 = whole(gen, x0.shape, 3, HF)
    y0, y1 = whole(gen, (60, 64), 3, BF), whole(gen, (60, 64), 3, BF)
    z0, z1 = (torch.randn((200, 32), generator=gen, device="cuda") for _ in range(2))
    pos, w = torch.arange(60, device="cuda").int().view(30, 2), torch.ones((30, 2), device="cuda")
    offsets = torch.tensor([0, 30], dtype=torch.int32, device="cuda")
    busy = torch.randn((4096, 4096), generator=gen, device="cuda")
    calls = {
        "project": (x0, x1, lambda x: p.project(x, W, adapter, A, B, scale, stream=stream),
                    lambda got: exact(got, plain_project(x1, W, adapter, A, B, scale))),
        "route": (z0, z1, lambda z: p.route(z, 3, stream=stream)[0],
                  lambda got: torch.testing.assert_close(got.long(), z1.topk(3).indices, rtol=0, atol=0)),
        "expert_project": (x0, x1, lambda x: p.expert_project(x, W[None], offsets, stream=stream),
                           lambda got: exact(got, plain_project(x1, W))),
        "expert_combine": (y0, y1, lambda y: p.expert_combine(y, pos, w, stream=stream),
                           lambda got: exact(got, y1.double().view(30, 2, 64).sum(1))),
    }
    for name, (old, new, call, check) in calls.items():
        given, written = old.clone(), torch.cuda.Event()
        call(given)  # (whatever a first call sets up)
        torch.cuda.synchronize()
        with torch.cuda.stream(s):
            for _ in range(50):  # tens of milliseconds
                torch.mm(busy, busy)
            given.copy_(new)
            written.record(s)
        got = call(given)
        assert not written.query(), name  # the call was made before its input was there
        torch.cuda.synchronize()
        check(got)


GUARD = 1 << 16


def guarded(size):
    """`size` bytes between two guards, and whether those are as they were."""
    all_ = torch.full((2 * GUARD + size,), 0xa5, dtype=torch.uint8, device="cuda")
    return all_[GUARD:GUARD + size], lambda: bool((all_[:GUARD] == 0xa5).all()) and bool((all_[GUARD + size:] == 0xa5).all())


@pytest.mark.parametrize("dtype", [BF, HF], ids=["bf16", "fp16"])
@pytest.mark.parametrize("T,K,N,rank,adapters", [
    (25, 2560, 320, 32, 6), (17, 520, 127, 128, 3), (32, 10240, 66, 8, 2),  # v and its splits
    (333, 10240, 2560, 64, 16), (333, 10240, 2560, 0, 0), (45, 8720, 4215, 16, 4), (600, 10240, 700, 40, 4),  # tiles, splits of K
    (1801, 2528, 2429, 16, 5), (2786, 8208, 399, 8, 3), (2479, 3816, 1843, 0, 0), (810, 4080, 3163, 24, 4),  # wide ones
    (3001, 128, 4099, 16, 2), (4097, 320, 2900, 128, 30),  # pieces of v
    (6600, 2568, 2560, 16, 6), (6600, 2568, 2560, 0, 0), (8193, 264, 10240, 8, 4),  # in two parts
])
def test_project_stays_inside_its_scratch(p, T, K, N, rank, adapters, dtype):
    case("project scratch", T, K, N, rank, adapters, dtype)
    x, W, adapter, A, B, scale = project_inputs(T, K, N, dtype, rank, adapters)
    lib = p.library()
    size = lib.hc_project_work(T, K, N, rank)
    work, untouched = guarded(size)
    out = torch.empty((T, N), dtype=F4, device="cuda")
    ptr = lambda t: None if t is None else t.data_ptr()  # noqa: E731
    for short in {0, min(size, 1)}:
        status = lib.hc_project(T, K, N, p._TYPE[dtype], x.data_ptr(), K, W.data_ptr(), ptr(adapter), adapters, rank,
                                ptr(A), ptr(B), ptr(scale), out.data_ptr(), N, p.HC_FP32, work.data_ptr(), size - short,
                                torch.cuda.current_stream().cuda_stream)
        assert (status == p.HC_OK) == (short == 0)
    assert untouched()
    exact(out, plain_project(x, W, adapter, A, B, scale))


@pytest.mark.parametrize("T,E,k", [(129, 64, 8), (257, 60, 8), (300, 257, 7), (4097, 64, 8), (8200, 256, 17), (33000, 40, 2)])
def test_route_stays_inside_its_scratch_and_outputs(p, T, E, k):
    case("route scratch", T, E, k)
    z = torch.randn((T, E), generator=new_gen(T), device="cuda")
    lib = p.library()
    size = lib.hc_route_work(T, E, k)
    assert size > 0
    parts = [guarded(n) for n in (4 * T * k, 4 * T * k, 4 * (E + 1), 4 * T * k, 4 * T * k, size)]
    assert lib.hc_route(T, E, k, z.data_ptr(), E, p.HC_FP32, 1, *[part.data_ptr() for part, _ in parts], size,
                        torch.cuda.current_stream().cuda_stream) == p.HC_OK
    assert all(untouched() for _, untouched in parts)
    for got, want in zip((part for part, _ in parts), p.route(z, k)):
        assert torch.equal(got.view(want.dtype), want.flatten())
