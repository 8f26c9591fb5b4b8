"""The attention between the projections on an MI355X, through the binding,
against plain 64-bit forms of its definitions.

Caches are paged in a random order, and what no request holds of them, the rest
of a last page too, is NaN.  Bounds are derived where they are used, from the
half step of a rounding (bf16 2^-8, fp16 2^-11, fp32 2^-24, relative)."""
import math

import pytest
import torch

pytestmark = pytest.mark.gpu

BF, HF, F4 = torch.bfloat16, torch.float16, torch.float32
TYPES = pytest.mark.parametrize("dtype", [BF, HF], ids=["bf16", "fp16"])
NAN = float("nan")


@pytest.fixture(scope="module")
def a():
    from hyper_connection_residual_amd import attention
    assert torch.cuda.is_available()
    return attention


def case(*what):
    print("case:", *what, flush=True)


def new_gen(seed):
    gen = torch.Generator(device="cuda")
    gen.manual_seed(seed)
    return gen


def ints(x):
    return torch.tensor(x, dtype=torch.int32, device="cuda")


class Call:
    """A batch of requests [(new tokens, length)], their cache (random pages, NaN where nothing is) and queries."""

    def __init__(self, a, requests, Hq, Hkv, D, page, dtype, seed=0, prefixes=(), starts=None, sigma=2.5, width=None):
        gen = new_gen(seed)
        host = torch.Generator().manual_seed(seed)
        self.a, self.requests, self.prefixes, self.dtype = a, requests, list(prefixes), dtype
        new, lengths = [n for n, _ in requests], [L for _, L in requests]
        self.T, self.Hq, self.Hkv, self.D, self.page = sum(new), Hq, Hkv, D, page
        need = [-(-L // page) for L in lengths + self.prefixes]
        pages = sum(need) + 3
        order = torch.randperm(pages, generator=host, dtype=torch.int32)
        self.keys = torch.full((pages, page, Hkv, D), NAN, dtype=dtype, device="cuda")
        self.values = self.keys.clone()
        rows, at = [], 0
        for L, k in zip(lengths + self.prefixes, need):
            mine = order[at:at + k].tolist()
            at += k
            rows.append(mine)
            for i, p in enumerate(mine):
                here = min(page, L - i * page)
                self.keys[p, :here] = torch.randn((here, Hkv, D), generator=gen, device="cuda").to(dtype)
                self.values[p, :here] = torch.randn((here, Hkv, D), generator=gen, device="cuda").to(dtype)
        # entries past a request's pages: pages that no one may read
        w = width or max(1, max(need))
        table = ints([r + [-7 if i % 2 else 1 << 30 for i in range(w - len(r))] for r in rows])
        off = [0]
        for n in new:
            off.append(off[-1] + n)
        self.offsets, self.lengths, self.table = ints(off), ints(lengths), table[:len(new)].contiguous()
        self.off = off
        self.q = (sigma * torch.randn((self.T, Hq, D), generator=gen, device="cuda")).to(dtype)
        self.cache, self.batch = a.PagedCache(self.keys, self.values), a.Batch(self.offsets, self.lengths, self.table)
        self.starts = starts
        if self.prefixes:
            self.prefix_table = table[len(new):].contiguous()
            self.prefix = a.SharedPrefix(ints(starts), ints(self.prefixes), self.prefix_table)
        self.scale = D ** -0.5

    def group(self, b):
        for g in range(len(self.prefixes)):
            if self.starts[g] <= b < self.starts[g + 1]:
                return g
        return None

    def sequence(self, b, x):
        """Request b's positions of the cache x, [L, Hkv, D] in 64 bits."""
        def rows(row, L):
            j = torch.arange(L, device="cuda")
            return x[row.long()[j // self.page], j % self.page].double()
        own = rows(self.table[b], self.requests[b][1])
        g = self.group(b)
        return own if g is None else torch.cat([rows(self.prefix_table[g], self.prefixes[g]), own])

    def positions(self, b):
        n, L = self.requests[b]
        g = self.group(b)
        before = 0 if g is None else self.prefixes[g]
        return torch.arange(before + L - n, before + L, device="cuda")

    def want(self, cap=0.0, slopes=None, first=None, last=None, keys=None, values=None):
        """(results, the same of the values' magnitudes, the scores' error bound), in 64 bits."""
        out = torch.zeros((self.T, self.Hq, self.D), dtype=torch.float64, device="cuda")
        size, error = out.clone(), torch.zeros((self.T, self.Hq), dtype=torch.float64, device="cuda")
        G = self.Hq // self.Hkv
        for b, (n, _) in enumerate(self.requests):
            if n == 0:
                continue
            t = slice(self.off[b], self.off[b + 1])
            k, v = self.sequence(b, self.keys if keys is None else keys), self.sequence(b, self.values if values is None else values)
            p, j = self.positions(b), torch.arange(k.shape[0], device="cuda")
            lo = torch.zeros_like(p) if first is None else first[t].long()
            hi = p + 1 if last is None else last[t].long()
            seen = (j >= lo[:, None]) & (j < hi[:, None])
            for h in range(self.Hq):
                q = self.q[t, h].double()
                z = q @ k[:, h // G].T * self.scale
                # an fp32 sum of D products: D steps of 2^-23 (the matrix cores need not round to nearest) of their
                # magnitudes; scaling, cap, bias and the maximum's subtraction: 8 roundings of what they are made of
                size_of = (q.abs() @ k[:, h // G].abs().T) * abs(self.scale)
                e = (self.D + 8) * 2.0 ** -23 * size_of
                if cap:
                    z = cap * torch.tanh(z / cap)
                    e = e + 16 * 2.0 ** -23 * cap
                if slopes is not None:
                    bias = slopes[h].double() * (p[:, None] - j).abs()
                    z = z - bias
                    e = e + 8 * 2.0 ** -23 * bias.abs()
                z = z.masked_fill(~seen, -math.inf)
                e = torch.where(seen & (z > z.amax(1, keepdim=True) - 40), e, 0.0)
                some = seen.any(1)
                w = torch.softmax(z[some], 1)
                clean = torch.where(torch.isfinite(v[:, h // G]), v[:, h // G], 0.0)
                rows = out[t, h]
                rows[some] = w @ clean
                out[t, h] = rows
                rows = size[t, h]
                rows[some] = w @ clean.abs()
                size[t, h] = rows
                error[t, h] = e.amax(1)
        return out, size, error

    def bound(self, want):
        """|got - want| within: the numerators' rounding (u of each) and their relative error (the scores' error and the
        exponential's, 8 2^-23), in sum and weights: twice; their sums' order, n 2^-23 twice; fp16 numerators under
        2^-14, 2^-25 each of up to n, at most the largest value; the output's rounding."""
        out, size, error = want
        u = torch.finfo(self.dtype).eps / 2
        n = max(L for _, L in self.requests) + max(self.prefixes, default=0)
        bound = (u + 2 * torch.expm1(error)[..., None] + (2 * n + 32) * 2.0 ** -23) * size + u * out.abs()
        if self.dtype == HF:
            top = torch.nan_to_num(self.values.float().abs(), nan=0.0, posinf=0.0).max().double()
            bound = bound + 2.0 ** -25 * (1 + n * top)
        return bound

    def check(self, got, want):
        out, size, _ = want
        u, bound = torch.finfo(self.dtype).eps / 2, self.bound(want)
        bad = ~((got.double() - out).abs() <= bound)
        assert not bool(bad.any()), (int(bad.sum()), bad.nonzero()[:4].tolist(), float(((got.double() - out).abs() / bound).nan_to_num(99).max()))
        # and far nearer than that on the whole: the numerators' and the output's roundings
        some = float(out.norm())
        if some:
            print("relative error", float((got.double() - out).norm()) / some, flush=True)
            assert float((got.double() - out).norm()) <= 1.5 * u * float(size.norm()) + 1e-6 * some


BATCHES = {
    "token": [(1, 1)],
    "token page": [(1, 16)],
    "token past page": [(1, 17)],
    "token long": [(1, 4097)],
    "decode": [(1, 33), (1, 700), (1, 1), (1, 2048), (1, 64), (1, 31), (1, 32), (1, 1500)],
    "decode some empty": [(0, 40), (1, 129), (0, 0), (1, 5), (1, 1000), (0, 7)],
    "windows": [(3, 100), (5, 5), (1, 900), (8, 1000), (2, 33)],
    "windows 16": [(16, 300), (9, 41), (16, 16)],
    "prompt": [(300, 300)],
    "prompt with past": [(130, 1531)],
    "mixed": [(1, 500), (257, 257), (1, 3), (40, 640), (0, 12), (7, 77)],
}
HEADS = [(4, 4, 64, 16), (5, 1, 128, 16), (8, 2, 256, 32), (6, 3, 80, 64), (8, 1, 40, 16), (4, 2, 136, 128), (2, 2, 8, 16), (20, 4, 128, 256)]


@TYPES
@pytest.mark.parametrize("name", BATCHES)
@pytest.mark.parametrize("Hq,Hkv,D,page", HEADS)
def test_attend(a, name, Hq, Hkv, D, page, dtype):
    case("attend", name, Hq, Hkv, D, page, dtype)
    c = Call(a, BATCHES[name], Hq, Hkv, D, page, dtype, seed=len(name))
    c.check(a.attend(c.q, c.cache, c.batch), c.want())


def ranges(c, kind, seed=5):
    """first and last of every token: windows, packed documents, prefixes, or any, some of them empty."""
    host = torch.Generator().manual_seed(seed)
    first, last = [], []
    for b in range(len(c.requests)):
        p = c.positions(b).cpu()
        L = int(c.sequence(b, c.keys).shape[0])
        lo, hi = torch.zeros_like(p), p + 1
        if kind == "window":
            lo = p - 37
        elif kind == "documents":
            starts = torch.cat([torch.zeros(1, dtype=torch.int64), torch.randint(0, L + 1, (1 + L // 60,), generator=host)]).sort().values
            lo = starts[torch.searchsorted(starts, p, right=True) - 1]
        elif kind == "prefix":
            hi = torch.maximum(hi, torch.tensor(int(0.6 * L)))
        elif kind == "all":
            hi = torch.full_like(p, L)
        elif kind == "any":
            lo = torch.randint(-5, L + 9, p.shape, generator=host)
            hi = torch.randint(-5, L + 9, p.shape, generator=host)
        first.append(lo)
        last.append(hi)
    first, last = (torch.cat(x).int().cuda() for x in (first, last))
    return {"window": (first, None), "documents": (first, None), "prefix": (None, last), "all": (None, last), "any": (first, last)}[kind]


@TYPES
@pytest.mark.parametrize("kind", ["window", "documents", "prefix", "all", "any"])
@pytest.mark.parametrize("name,Hq,Hkv,D,page", [("decode", 5, 1, 128, 16), ("windows", 4, 2, 64, 16), ("windows 16", 8, 2, 256, 32), ("mixed", 4, 4, 128, 16), ("prompt with past", 6, 2, 72, 64), ("mixed", 6, 1, 256, 32),
                                                ("windows 16", 8, 1, 64, 16), ("decode", 40, 1, 128, 16)])
def test_attend_masks(a, name, Hq, Hkv, D, page, kind, dtype):
    case("masks", name, Hq, Hkv, D, page, kind, dtype)
    c = Call(a, BATCHES[name], Hq, Hkv, D, page, dtype, seed=3)
    first, last = ranges(c, kind)
    got = a.attend(c.q, c.cache, c.batch, first=first, last=last)
    want = c.want(first=first, last=last)
    c.check(got, want)
    if kind == "any":  # tokens that see nothing
        lo, hi = first.clone(), last.clone()
        for b in range(len(c.requests)):
            t = slice(c.off[b], c.off[b + 1])
            hi[t].clamp_(max=c.requests[b][1])
        none = lo.clamp(min=0) >= hi
        if name != "decode" or bool(none.any()):
            assert bool(none.any()) and bool((got[none] == 0).all())


@TYPES
@pytest.mark.parametrize("cap,bias", [(5.0, False), (50.0, False), (0.0, True), (8.0, True)])
@pytest.mark.parametrize("name,Hq,Hkv,D,page", [("decode", 5, 1, 128, 16), ("windows 16", 8, 2, 64, 16), ("mixed", 4, 4, 128, 16), ("windows", 4, 1, 256, 32), ("mixed", 6, 3, 96, 16)])
def test_attend_cap_and_bias(a, name, Hq, Hkv, D, page, cap, bias, dtype):
    case("cap and bias", name, Hq, Hkv, D, page, cap, bias, dtype)
    c = Call(a, BATCHES[name], Hq, Hkv, D, page, dtype, seed=4)
    slopes = torch.exp2(-torch.arange(1, Hq + 1, device="cuda") * 8.0 / Hq) if bias else None
    c.check(a.attend(c.q, c.cache, c.batch, cap=cap, slopes=slopes), c.want(cap=cap, slopes=slopes))
    last = ranges(c, "all")[1]  # later positions, too: the distance has no sign
    c.check(a.attend(c.q, c.cache, c.batch, cap=cap, slopes=slopes, last=last), c.want(cap=cap, slopes=slopes, last=last))


@TYPES
@pytest.mark.parametrize("scale,cap", [(0.0, 0.0), (-0.125, 0.0), (-0.125, 4.0), (0.0, 4.0), (0.125, 1e6), (0.125, 1e30), (0.125, 1e-6), (1e-42, 0.0)])
@pytest.mark.parametrize("name,Hq,Hkv,D,page", [("decode", 5, 1, 128, 16), ("windows 16", 8, 2, 64, 16), ("mixed", 4, 4, 128, 16), ("mixed", 6, 3, 96, 16), ("prompt", 4, 1, 256, 32), ("prompt", 5, 1, 128, 16)])
def test_attend_scales_and_caps_of_any_size(a, name, Hq, Hkv, D, page, scale, cap, dtype):
    case("scales", name, Hq, Hkv, D, page, scale, cap, dtype)
    c = Call(a, BATCHES[name], Hq, Hkv, D, page, dtype, seed=12)
    c.scale = scale
    got = a.attend(c.q, c.cache, c.batch, scale=scale, cap=cap)
    # Scores (up to about 30) that are far below the cap are as good as without one: its tanh adds 6 roundings of the score,
    # and the bound without a cap has D + 8 of what the score is made of.
    c.check(got, c.want(cap=0.0 if cap > 1e3 else cap))


MANY = {
    "2048 tokens": [(1, 1 + b % 50) for b in range(2048)],
    "2048 of some": [(b % 3, 3 + b % 70) for b in range(2048)],
    "100 of tiles": [(30 + b % 7, 40 + b) for b in range(100)],
    "70 of tiles": [(90, 95 + b) for b in range(70)],
    "long and short": [(1, 40)] * 200 + [(700, 900)] + [(2, 5)] * 100,
}


@pytest.mark.parametrize("name", MANY)
@pytest.mark.parametrize("Hq,Hkv,D,page", [(2, 2, 64, 16), (5, 1, 128, 16), (2, 1, 256, 32)])
def test_attend_many_requests(a, name, Hq, Hkv, D, page):
    case("many", name, Hq, Hkv, D, page)
    c = Call(a, MANY[name], Hq, Hkv, D, page, BF, seed=13)
    c.check(a.attend(c.q, c.cache, c.batch), c.want())


def test_attend_the_most_rows(a):
    """HC_MAX_ROWS rows: 4096 tokens of 64 heads; some of them against the formula."""
    case("most rows")
    c = Call(a, [(1000, 1000), (3096, 3100)], 64, 1, 64, 64, BF, seed=14)
    got = a.attend(c.q, c.cache, c.batch)
    some = Call(a, [(1000, 1000), (3096, 3100)], 64, 1, 64, 64, BF, seed=14)
    some.Hq, heads = 2, [0, 63]
    some.q = c.q[:, heads].contiguous()
    some.check(got[:, heads], some.want())
    with pytest.raises(ValueError):
        a.attend(c.q.repeat(2, 1, 1)[:4097], c.cache, c.batch)


@TYPES
@pytest.mark.parametrize("name", ["token long", "decode", "windows", "windows 16", "mixed", "prompt with past"])
@pytest.mark.parametrize("Hq,Hkv,D,page", [(4, 2, 64, 16), (5, 1, 128, 32), (2, 1, 256, 16), (8, 1, 104, 16)])
def test_attend_picks_the_one_position(a, name, Hq, Hkv, D, page, dtype):
    """Keys of -1 and 1 and queries 64 times one of them: all other scores are lower by far more than the exponential's
    range, and the result is that position's value, bit for bit."""
    case("pick", name, Hq, Hkv, D, page, dtype)
    c = Call(a, BATCHES[name], Hq, Hkv, D, page, dtype, seed=6)
    c.keys.copy_(c.keys.sign())  # (NaN stays)
    want = torch.empty_like(c.q)
    host = torch.Generator().manual_seed(1)
    for b, (n, L) in enumerate(c.requests):
        k, v = c.sequence(b, c.keys), c.sequence(b, c.values)
        for i in range(n):
            for h in range(Hq):
                j = int(torch.randint(0, L - n + i + 1, (), generator=host))
                c.q[c.off[b] + i, h] = (64 * k[j, h * Hkv // Hq]).to(dtype)
                want[c.off[b] + i, h] = v[j, h * Hkv // Hq].to(dtype)
    # (the largest product is 64 D; another key that agrees in all but one column is 128 lower, times this scale)
    assert torch.equal(a.attend(c.q, c.cache, c.batch, scale=2.0), want)


@TYPES
@pytest.mark.parametrize("name,Hq,Hkv,D,page", [("token long", 4, 1, 128, 16), ("decode", 4, 2, 128, 16), ("windows 16", 8, 2, 64, 32), ("windows", 2, 2, 256, 16), ("mixed", 4, 1, 128, 16), ("prompt", 6, 2, 80, 16)])
def test_attend_what_is_not_seen_does_not_matter(a, name, Hq, Hkv, D, page, dtype):
    """NaN and infinities in positions that a token does not see, of its own request and of others: not a bit changes.
    Infinite and NaN values of positions that it does see reach it."""
    case("not seen", name, Hq, Hkv, D, page, dtype)
    c = Call(a, BATCHES[name], Hq, Hkv, D, page, dtype, seed=7, sigma=0.5)
    want = a.attend(c.q, c.cache, c.batch)
    for b, (n, L) in enumerate(c.requests):
        if n < 1:
            continue
        # the last token's position, then a middle new one's, for keys and values
        for j in {L - 1, L - (n + 1) // 2}:
            at = int(c.table[b, j // page]), j % page
            for x, bad in ((c.values, NAN), (c.values, math.inf), (c.values, -math.inf), (c.keys, NAN)):
                kept = x[at].clone()
                x[at] = bad
                got = a.attend(c.q, c.cache, c.batch)
                x[at] = kept
                sees = torch.zeros(c.T, dtype=torch.bool, device="cuda")
                sees[c.off[b] + (j - (L - n)):c.off[b + 1]] = True
                assert torch.equal(got[~sees], want[~sees]), (b, j, bad)
                if x is c.values:
                    assert bool((torch.isnan(got[sees]) if math.isnan(bad) else got[sees] == bad).all()), (b, j, bad)
                else:
                    assert bool(torch.isnan(got[sees]).all())
    # a token's own query
    bad = c.q.clone()
    t = c.T // 2
    c.q[t] = NAN
    got = a.attend(c.q, c.cache, c.batch)
    c.q.copy_(bad)
    assert bool(torch.isnan(got[t]).all())
    got[t] = want[t]
    assert torch.equal(got, want)


@TYPES
@pytest.mark.parametrize("name", ["decode", "windows 16", "mixed"])
def test_attend_layouts(a, name, dtype):
    """Queries and results as columns of wider rows; heads before rows, keys and values of one tensor, in the cache."""
    case("layouts", name, dtype)
    c = Call(a, BATCHES[name], 6, 2, 64, 16, dtype, seed=8)
    want = a.attend(c.q, c.cache, c.batch)
    wide = torch.full((c.T, 8, 80), NAN, dtype=dtype, device="cuda")
    wide[:, 1:7, 8:72] = c.q
    out = torch.full((c.T + 2, 7, 72), 7.0, dtype=dtype, device="cuda")
    to = out[1:-1, 1:, :64]
    assert a.attend(wide[:, 1:7, 8:72], c.cache, c.batch, out=to).data_ptr() == to.data_ptr()
    assert torch.equal(to, want)
    to.fill_(7.0)
    assert bool((out == 7).all())
    by_head = [x.transpose(1, 2).contiguous().transpose(1, 2) for x in (c.keys, c.values)]
    assert torch.equal(a.attend(c.q, a.PagedCache(*by_head), c.batch), want)
    both = torch.full((c.keys.shape[0], 2, 16, 2, 72), NAN, dtype=dtype, device="cuda")
    both[:, 0, :, :, :64], both[:, 1, :, :, :64] = c.keys, c.values
    assert torch.equal(a.attend(c.q, a.PagedCache(both[:, 0, :, :, :64], both[:, 1, :, :, :64]), c.batch), want)
    table = torch.full((len(c.requests), c.table.shape[1] + 5), -1, dtype=torch.int32, device="cuda")
    table[:, 2:-3] = c.table
    assert torch.equal(a.attend(c.q, c.cache, a.Batch(c.offsets, c.lengths, table[:, 2:-3])), want)


@pytest.mark.parametrize("Hq", [2, 10, 40])
def test_attend_tokens_of_no_request_are_left_alone(a, Hq):
    case("no request", Hq)
    for T, off in ((9, [0, 3, 5]), (9, [2, 3, 9]), (300, [10, 150, 290]), (300, [300, 300, 300]), (40, [0, 0, 0])):
        c = Call(a, [(off[1] - off[0], 400), (off[2] - off[1], 300)], Hq, 2, 64, 16, BF)
        q = torch.randn((T, Hq, 64), generator=new_gen(2), device="cuda").to(BF)
        q[off[0]:off[2]] = c.q
        out = torch.full_like(q, 7.0)
        a.attend(q, c.cache, a.Batch(ints(off), c.lengths, c.table), out=out)
        c.check(out[off[0]:off[2]], c.want()) if c.T else None
        out[off[0]:off[2]] = 7.0
        assert bool((out == 7).all())


@pytest.mark.parametrize("Hq", [2, 10, 40])
def test_attend_lists_that_do_not_fit(a, Hq):
    """Offsets past the tokens and out of order, lengths past the table and below zero, pages that the cache does not
    have: read as zeros, nothing outside the output is written, and the other requests' results stay."""
    case("lists", Hq)
    c = Call(a, [(2, 100), (3, 70), (60, 200), (1, 40)], Hq, 2, 128, 16, BF)
    want = c.want()

    def others(got, b):
        keep = torch.ones(c.T, dtype=torch.bool, device="cuda")
        keep[c.off[b]:c.off[b + 1]] = False
        return bool(((got.double() - want[0]).abs() <= c.bound(want))[keep].all())

    for b, length in ((0, 1 << 30), (0, 2 ** 31 - 1), (2, -5), (2, -2 ** 31), (1, 0), (2, 20), (3, 41)):
        lengths = c.lengths.clone()
        lengths[b] = length
        got = a.attend(c.q, c.cache, a.Batch(c.offsets, lengths, c.table))
        assert others(got, b), length
        if length <= 0:
            assert bool((got[c.off[b]:c.off[b + 1]] == 0).all())
        if length == 20:  # the last 20 of its 60 tokens have positions
            assert bool((got[c.off[2]:c.off[2] + 40] == 0).all()) and bool((got[c.off[2] + 40:c.off[3]] != 0).any(-1).all())
    for page in (-1, -2 ** 31, c.keys.shape[0], 2 ** 31 - 1):
        for b in range(4):
            table = c.table.clone()
            table[b, 1] = page
            got = a.attend(c.q, c.cache, a.Batch(c.offsets, c.lengths, table))
            assert others(got, b)
            # the page's 16 positions are zeros, keys and values
            keys, values = c.keys.clone(), c.values.clone()
            keys[c.table[b, 1]], values[c.table[b, 1]] = 0, 0
            right, size, error = c.want(keys=keys, values=values)
            mine = slice(c.off[b], c.off[b + 1])
            assert float((got.double() - right)[mine].norm()) <= 2.0 ** -7 * float(size[mine].norm())
    for off in ([0, 2, 5, 65, 1 << 30], [-9, 2, 5, 65, 66], [0, 60, 3, 40, 66], [66, 0, 66, 0, 66], [2 ** 31 - 1, -2 ** 31, 5, 5, 5]):
        out = torch.full((c.T + 8, Hq, 128), 7.0, dtype=BF, device="cuda")
        a.attend(c.q, c.cache, a.Batch(ints(off), c.lengths, c.table), out=out[4:-4])
        torch.cuda.synchronize()
        assert bool((out[:4] == 7).all()) and bool((out[-4:] == 7).all())
    got = a.attend(c.q, c.cache, a.Batch(c.offsets, c.lengths, c.table[:, :0]))  # no pages at all
    assert bool((got == 0).all())


SHARED = [
    # requests, prefixes, starts
    ([(1, 1)], [1], [0, 1]),
    ([(1, 30), (1, 200), (1, 1)], [700], [0, 3]),
    ([(1, 5)] * 40, [2000], [0, 40]),
    ([(3, 40), (1, 7), (8, 300), (2, 2), (1, 90)], [333, 17], [0, 2, 5]),
    ([(1, 50), (2, 20), (1, 700), (0, 30), (4, 64)], [128, 1, 500], [1, 2, 2, 4]),  # requests without, prefixes without
    ([(150, 150), (1, 40), (33, 60)], [257], [0, 3]),
    ([(1, 50)] * 3, [0], [0, 3]),
    ([(1, 60)] * 70, [3000, 100], [0, 50, 70]),
]


@TYPES
@pytest.mark.parametrize("Hq,Hkv,D,page", [(4, 4, 64, 16), (5, 1, 128, 16), (4, 2, 256, 32), (6, 2, 80, 64), (20, 2, 128, 16)])
@pytest.mark.parametrize("layout", range(len(SHARED)))
def test_attend_shared(a, layout, Hq, Hkv, D, page, dtype):
    case("shared", layout, Hq, Hkv, D, page, dtype)
    requests, prefixes, starts = SHARED[layout]
    c = Call(a, requests, Hq, Hkv, D, page, dtype, seed=9, prefixes=prefixes, starts=starts)
    c.check(a.attend_shared(c.q, c.cache, c.batch, c.prefix), c.want())


@TYPES
@pytest.mark.parametrize("kind", ["window", "documents", "prefix", "any"])
def test_attend_shared_masks_cap_and_bias(a, kind, dtype):
    case("shared masks", kind, dtype)
    requests, prefixes, starts = SHARED[4]
    c = Call(a, requests, 6, 2, 64, 16, dtype, seed=10, prefixes=prefixes, starts=starts)
    first, last = ranges(c, kind)
    slopes = torch.tensor([0.5, 0.25, 0.1, 0.05, 0.01, 0.0], device="cuda")
    got = a.attend_shared(c.q, c.cache, c.batch, c.prefix, cap=20.0, slopes=slopes, first=first, last=last)
    c.check(got, c.want(cap=20.0, slopes=slopes, first=first, last=last))


@TYPES
def test_attend_shared_is_attend_over_the_whole(a, dtype):
    """The prefix's pages in every request's own table: the same sequences, in one segment."""
    case("shared and whole", dtype)
    c = Call(a, [(1, 40), (3, 130), (1, 16)], 4, 2, 128, 16, dtype, seed=11, prefixes=[320], starts=[0, 3])
    got = a.attend_shared(c.q, c.cache, c.batch, c.prefix)
    table = torch.cat([c.prefix_table.expand(3, -1), c.table], 1).contiguous()  # (320 is whole pages)
    whole = a.attend(c.q, c.cache, a.Batch(c.offsets, c.lengths + 320, table))
    assert float((got.double() - whole.double()).norm()) <= 2.0 ** (-7 if dtype == BF else -10) * float(whole.double().norm())


def test_attend_shared_lists_that_do_not_fit(a):
    case("shared lists")
    c = Call(a, [(1, 40), (3, 130), (1, 16)], 4, 2, 128, 16, BF, seed=12, prefixes=[320, 50], starts=[0, 2, 3])
    for starts, lengths, page in (([0, 2, 1 << 30], [320, 50], None), ([-4, 2, 3], [320, 50], None), ([2, 0, 3], [320, 50], None),
                                  ([0, 2, 3], [1 << 30, -4], None), ([0, 2, 3], [320, 50], -1), ([0, 2, 3], [320, 50], 1 << 30), ([3, 3, 3], [320, 50], None),
                                  ([0, 0, 0], [0, 0], None)):
        table = c.prefix_table.clone()
        if page is not None:
            table[0, 3] = page
        out = torch.full((c.T + 8, 4, 128), 7.0, dtype=BF, device="cuda")
        a.attend_shared(c.q, c.cache, c.batch, a.SharedPrefix(ints(starts), ints(lengths), table), out=out[4:-4])
        torch.cuda.synchronize()
        assert bool((out[:4] == 7).all()) and bool((out[-4:] == 7).all())


def plain_turned(x, positions, f, weight, eps, interleaved):
    x = x.double()
    if weight is not None:
        x = x / torch.sqrt((x * x).mean(-1, keepdim=True) + eps) * weight.double()
    if f is None:
        return x
    n = f.numel()
    y, angle = x.clone(), positions.double()[:, None, None] * f.double()
    first, second = (slice(0, 2 * n, 2), slice(1, 2 * n, 2)) if interleaved else (slice(0, n), slice(n, 2 * n))
    y[..., first] = x[..., first] * torch.cos(angle) - x[..., second] * torch.sin(angle)
    y[..., second] = x[..., second] * torch.cos(angle) + x[..., first] * torch.sin(angle)
    return y


def check_turned(got, x, positions, f, weight, eps, interleaved):
    """The norm: D sums, a root, a division and two products, (D / 2 + 4) 2^-23; sines and cosines within 2^-21 of the
    exact angle's; two products and a sum; the rounding of the output."""
    want = plain_turned(x, positions, f, weight, eps, interleaved)
    plain = plain_turned(x, positions, None, weight, eps, interleaved).abs()
    size = plain.clone()
    if f is not None:
        n = f.numel()
        first, second = (slice(0, 2 * n, 2), slice(1, 2 * n, 2)) if interleaved else (slice(0, n), slice(n, 2 * n))
        size[..., first] = size[..., second] = plain[..., first] + plain[..., second]
    u = torch.finfo(got.dtype).eps / 2
    tiny = 2.0 ** -25 if got.dtype == HF else 0.0
    bound = u * want.abs() + ((x.shape[-1] / 2 + 8) * 2.0 ** -23 + 2.0 ** -21) * size + tiny
    bad = ~((got.double() - want).abs() <= bound)
    assert not bool(bad.any()), (int(bad.sum()), bad.nonzero()[:4].tolist())


ROTATIONS = [(64, 64, False), (128, 128, False), (256, 256, False), (256, 64, True), (80, 32, False), (96, 96, True), (8, 8, True), (8, 8, False), (40, 24, False), (136, 72, False), (128, 0, False),
             (200, 200, True), (248, 248, False)]


@TYPES
@pytest.mark.parametrize("weighted", [False, True])
@pytest.mark.parametrize("T,H", [(1, 1), (3, 5), (8, 20), (1000, 7), (9000, 3)])
@pytest.mark.parametrize("D,R,interleaved", ROTATIONS)
def test_rotate_heads(a, T, H, D, R, interleaved, weighted, dtype):
    case("rotate", T, H, D, R, interleaved, weighted, dtype)
    gen = new_gen(T + H + D)
    x = (3.0 * torch.randn((T, H, D), generator=gen, device="cuda")).to(dtype)
    f = (10000.0 ** (-torch.arange(0, R, 2, device="cuda") / R)).float() if R else None
    positions = torch.randint(0, 2 ** 20, (T,), generator=gen, device="cuda", dtype=torch.int32)
    positions[0] = 2 ** 31 - 1
    positions[-1] = -77 if T > 1 else 2 ** 31 - 1
    weight = 1.0 + 0.3 * torch.randn((D,), generator=gen, device="cuda") if weighted else None
    got = a.rotate_heads(x, positions, f, weight=weight, eps=1e-5, interleaved=interleaved)
    check_turned(got, x, positions, f, weight, 1e-5, interleaved)
    wide = torch.full((T, H + 1, D + 16), NAN, dtype=dtype, device="cuda")
    wide[:, :H, 8:D + 8] = x
    view = wide[:, :H, 8:D + 8]
    assert a.rotate_heads(view, positions, f, weight=weight, eps=1e-5, interleaved=interleaved, out=view) is view
    assert torch.equal(view, got)
    view.fill_(NAN)
    assert bool(torch.isnan(wide).all())


def test_rotate_heads_keeps_what_does_not_turn(a):
    case("rotate passes")
    x = torch.randn((30, 4, 128), generator=new_gen(1), device="cuda").to(BF)
    assert torch.equal(a.rotate_heads(x), x)
    zero = torch.zeros(30, dtype=torch.int32, device="cuda")
    f = torch.rand(32, generator=new_gen(2), device="cuda")
    assert torch.equal(a.rotate_heads(x, zero, f), x)
    y = a.rotate_heads(x, zero + 9, f)
    assert torch.equal(y[..., 64:], x[..., 64:]) and not torch.equal(y[..., :64], x[..., :64])
    x[3, 2, 5] = NAN  # a head's NaN stays in its pair, or with a norm in its head
    z = a.rotate_heads(x, zero + 9, f)
    assert int(torch.isnan(z).sum()) == 2 and bool(torch.isnan(z[3, 2, 5])) and bool(torch.isnan(z[3, 2, 37]))
    z = a.rotate_heads(x, zero + 9, f, weight=torch.ones(128, device="cuda"))
    assert bool(torch.isnan(z[3, 2]).all()) and int(torch.isnan(z).sum()) == 128
    nothing = torch.zeros((2, 3, 64), dtype=HF, device="cuda")  # a head of zeros stays one
    assert bool((a.rotate_heads(nothing, zero[:2], f, weight=torch.ones(64, device="cuda")) == 0).all())


APPENDS = {
    "token": [(1, 1)],
    "decode": [(1, 33), (1, 16), (1, 17), (1, 100)],
    "mixed": [(1, 5), (70, 300), (0, 9), (33, 33), (2, 31)],
    "prompts": [(900, 1000), (700, 700)],
    "many": [(1 + b % 3, 20 + b) for b in range(200)],
}


@TYPES
@pytest.mark.parametrize("name", APPENDS)
@pytest.mark.parametrize("Hq,Hkv,D,R,interleaved,page", [(20, 4, 128, 128, False, 16), (6, 3, 64, 64, True, 32), (8, 2, 80, 32, False, 16), (4, 1, 256, 256, False, 64), (3, 3, 24, 0, False, 16), (0, 2, 128, 64, False, 16)])
def test_append_heads(a, name, Hq, Hkv, D, R, interleaved, page, dtype):
    """The new tokens' keys and values are where attend will look for them, and nothing else of the cache changes."""
    case("append", name, Hq, Hkv, D, R, interleaved, page, dtype)
    c = Call(a, APPENDS[name], max(Hq, Hkv), Hkv, D, page, dtype, seed=13)
    gen = new_gen(14)
    rows = (2.0 * torch.randn((c.T, (Hq + 2 * Hkv) * D), generator=gen, device="cuda")).to(dtype)
    q, k, v = (x.unflatten(1, (-1, D)) for x in rows.split([Hq * D, Hkv * D, Hkv * D], dim=1)) if Hq else (None, *(
        x.unflatten(1, (-1, D)) for x in rows.split([Hkv * D, Hkv * D], dim=1)))
    f = (10000.0 ** (-torch.arange(0, R, 2, device="cuda") / R)).float() if R else None
    qw, kw = (1.0 + 0.2 * torch.randn((D,), generator=gen, device="cuda") for _ in range(2))
    for given, weights in ((None, (qw, kw)), (torch.randint(0, 10 ** 6, (c.T,), generator=gen, device="cuda", dtype=torch.int32), (None, kw))):
        keys, values = c.keys.clone(), c.values.clone()
        got = a.append_heads(q, k, v, a.PagedCache(keys, values), c.batch, f, positions=given, q_weight=weights[0], k_weight=weights[1],
                             interleaved=interleaved)
        where = [(b, i) for b, (n, L) in enumerate(c.requests) for i in range(L - n, L)]
        p = ints([i for _, i in where]) if given is None else given
        at = ints([int(x) for x in c.table[[b for b, _ in where], [i // page for _, i in where]].tolist()]).long(), ints([i % page for _, i in where]).long()
        check_turned(keys[at], k, p, f, weights[1], 1e-6, interleaved)
        assert torch.equal(values[at], v)
        if Hq:
            check_turned(got, q, p, f, weights[0], 1e-6, interleaved)
        else:
            assert got is None
        old_k, old_v = c.keys.clone(), c.values.clone()
        for x in (keys, values, old_k, old_v):
            x[at] = 0
        assert all(bool(((x == y) | (torch.isnan(x) & torch.isnan(y))).all()) for x, y in ((keys, old_k), (values, old_v)))


def test_append_heads_of_no_place(a):
    """Tokens of no request, of positions before 0 or past the table, on pages that the cache does not have."""
    case("append nowhere")
    c = Call(a, [(4, 40), (3, 20), (2, 64)], 4, 2, 64, 16, BF, seed=15)
    gen = new_gen(16)
    T = c.T + 5
    q, k, v = (torch.randn((T, h, 64), generator=gen, device="cuda").to(BF) for h in (4, 2, 2))
    kept = c.keys.clone(), c.values.clone()
    out = torch.full_like(q, 7.0)
    table = c.table.clone()
    table[2, 3] = 1 << 30
    lengths = ints([2, 16 * table.shape[1] + 3, 64])  # two of the first's four tokens have no position, none of the second's a page
    a.append_heads(q, k, v, c.cache, a.Batch(c.offsets, lengths, table), out=out)
    assert torch.equal(out[:c.T], q[:c.T]) and bool((out[c.T:] == 7).all())
    at = c.table[0, 0].long(), slice(0, 2)
    assert torch.equal(c.keys[at], k[2:4]) and torch.equal(c.values[at], v[2:4])
    c.keys[at], c.values[at] = kept[0][at], kept[1][at]
    for x, y in zip((c.keys, c.values), kept):
        assert bool(((x == y) | (torch.isnan(x) & torch.isnan(y))).all())
    for off in ([5, 0, 9, 3], [-4, 2, 1 << 30, 3], [2 ** 31 - 1] * 4):
        a.append_heads(q, k, v, c.cache, a.Batch(ints(off), c.lengths, c.table), out=out)
    torch.cuda.synchronize()


def test_nothing_to_do(a):
    case("empty")
    c = Call(a, [(0, 40), (0, 0)], 4, 2, 64, 16, BF)
    assert a.attend(c.q, c.cache, c.batch).shape == (0, 4, 64)
    assert a.rotate_heads(c.q).shape == (0, 4, 64)
    assert a.append_heads(c.q, c.q[:, :2], c.q[:, :2], c.cache, c.batch).shape == (0, 4, 64)
    q = torch.full((3, 4, 64), 7.0, dtype=BF, device="cuda")
    out = q.clone()
    a.attend(q, c.cache, c.batch, out=out)  # tokens, but of no request
    assert bool((out == 7).all())


def test_offsets_past_32_bits(a):
    """A cache of more than 2^32 bytes of keys, pages at its two ends, and queries and results past 2^31 elements' stride."""
    case("past 32 bits")
    pages, page, D = 150000, 64, 256  # 4.9 GB each
    gen = new_gen(17)
    keys, values = (torch.zeros((pages, page, 1, D), dtype=BF, device="cuda") for _ in range(2))
    table = ints([[pages - 1, 0, pages - 2, 77]])
    for T, L in ((1, 200), (150, 256)):
        keys[table[0].long()] = torch.randn((4, page, 1, D), generator=gen, device="cuda").to(BF)
        q, k, v = (torch.randn((T, h, D), generator=gen, device="cuda").to(BF) for h in (2, 1, 1))
        values[table[0].long()] = torch.randn((4, page, 1, D), generator=gen, device="cuda").to(BF)
        batch, cache = a.Batch(ints([0, T]), ints([L]), table), a.PagedCache(keys, values)
        a.append_heads(q, k, v, cache, batch)
        p = torch.arange(L - T, L, device="cuda")
        assert torch.equal(keys[table[0].long()[p // page], p % page], k) and torch.equal(values[table[0].long()[p // page], p % page], v)
        got = a.attend(q, cache, batch)
        j = torch.arange(L, device="cuda")
        kk, vv = (x[table[0].long()[j // page], j % page, 0].double() for x in (keys, values))
        z = (q.double() @ kk.T / 16).masked_fill(j > p[:, None, None], -math.inf)
        right = torch.softmax(z, -1) @ vv
        assert float((got.double() - right).norm()) <= 2.0 ** -7 * float(right.norm())
    del keys, values, cache
    # two tokens that lie 3 GB apart
    x = torch.zeros((3 << 30) // 2 + 4096, dtype=BF, device="cuda")
    far = x.as_strided((2, 2, 128), ((3 << 30) // 2, 128, 1))
    far.copy_(torch.randn((2, 2, 128), generator=gen, device="cuda"))
    c = Call(a, [(2, 90)], 2, 1, 128, 16, BF)
    want = a.attend(far.contiguous(), c.cache, c.batch)
    assert torch.equal(a.attend(far, c.cache, c.batch), want)
    out = torch.zeros_like(x).as_strided(far.shape, far.stride())
    assert torch.equal(a.attend(far, c.cache, c.batch, out=out), want)
    assert torch.equal(a.rotate_heads(far, out=out), far)


def layer(a, p, x, w, cache, batch, f, heads, prefix=None, positions=None):
    """A layer's attention on the read's image: projection, norms and rotation into the cache, attention, projection."""
    Hq, Hkv, D = heads
    rows = p.project(x, w["qkv"], *w["adapters"])
    q, k, v = (y.unflatten(1, (-1, D)) for y in rows.split([Hq * D, Hkv * D, Hkv * D], dim=1))
    q = a.append_heads(q, k, v, cache, batch, f, positions=positions, q_weight=w["q"], k_weight=w["k"])
    y = a.attend(q, cache, batch) if prefix is None else a.attend_shared(q, cache, batch, prefix)
    return p.project(y.flatten(1), w["out"], out_dtype=F4), (rows, q, y)


def layer_weights(gen, K, heads, T):
    Hq, Hkv, D = heads
    rand = lambda *s: (0.02 * torch.randn(s, generator=gen, device="cuda")).to(BF)  # noqa: E731
    N = (Hq + 2 * Hkv) * D
    return {"qkv": rand(N, K), "out": rand(K, Hq * D), "q": 1 + 0.1 * torch.randn((D,), generator=gen, device="cuda"),
            "k": 1 + 0.1 * torch.randn((D,), generator=gen, device="cuda"),
            "adapters": ((torch.arange(T, device="cuda") % 3 - 1).int(), rand(2, 16, K), rand(2, N, 16))}


@pytest.mark.parametrize("requests", [[(1, 300)], [(1, 40), (1, 700), (1, 9)], [(3, 90), (5, 5), (2, 400)], [(200, 260), (1, 50)]])
@pytest.mark.parametrize("shared", [False, True])
def test_read_project_append_attend_project_together(a, requests, shared):
    """As a layer runs them, on the read's image; every stage against its definition on the stage before, and the result
    as the next read's pending write."""
    from hyper_connection_residual_amd import binding, projections as p, workloads as wl
    T = sum(n for n, _ in requests)
    case("together", requests, shared)
    inp = wl.config_inputs(2, T=T)
    dev = lambda x: torch.from_numpy(x).cuda()  # noqa: E731
    R, w_norm = dev(inp.R), dev(inp.w_norm)
    Wd, Wu = dev(inp.W_down.view("int16")), dev(inp.W_up.view("int16"))
    _, x, _ = binding.read(R, w_norm, Wd, Wu, pending=dev(inp.pending))
    heads = (20, 5, 128)
    c = Call(a, requests, 20, 5, 128, 16, BF, seed=18, prefixes=[150] if shared else [], starts=[0, len(requests)])
    w = layer_weights(new_gen(T), 2560, heads, T)
    f = (10000.0 ** (-torch.arange(0, 128, 2, device="cuda") / 128)).float()
    positions = torch.cat([c.positions(b) for b in range(len(requests))]).int()
    out, (rows, q, y) = layer(a, p, x, w, c.cache, c.batch, f, heads, c.prefix if shared else None, positions if shared else None)
    check_turned(q, rows[:, :2560].unflatten(1, (20, 128)), positions, f, w["q"], 1e-6, False)
    for b, (n, L) in enumerate(requests):
        t = slice(c.off[b], c.off[b + 1])
        j = torch.arange(L - n, L, device="cuda")
        at = c.table[b].long()[j // 16], j % 16
        check_turned(c.keys[at], rows[t, 2560:-640].unflatten(1, (5, 128)), positions[t], f, w["k"], 1e-6, False)
        assert torch.equal(c.values[at].flatten(1), rows[t, -640:])
    c.q = q
    c.check(y, c.want())
    want = y.flatten(1).double() @ w["out"].double().T
    size = y.flatten(1).abs().double() @ w["out"].abs().double().T
    assert bool(((out.double() - want).abs() <= 2560 * 2.0 ** -23 * size).all())
    mixed, _, _ = binding.read(R, w_norm, Wd, Wu, pending=out[:, None, :].expand(T, 4, 2560).contiguous())
    assert bool(torch.isfinite(mixed).all())


@pytest.mark.parametrize("new", [1, 4, 60])
@pytest.mark.parametrize("shared", [False, True])
def test_captured_and_replayed(a, new, shared):
    """The layer in a graph, replayed for other inputs and lengths, with eager work between: every replay equals the
    eager result bit for bit."""
    from hyper_connection_residual_amd import projections as p
    case("graph", new, shared)
    requests = [(new, 200), (new, 130), (new, 64)]
    c = Call(a, requests, 4, 2, 64, 16, BF, seed=19, prefixes=[90] if shared else [], starts=[0, 3], width=20)
    c.keys.nan_to_num_(0.0)
    c.values.nan_to_num_(0.0)
    T, heads = c.T, (4, 2, 64)
    w, f = layer_weights(new_gen(20), 256, heads, T), torch.rand(32, generator=new_gen(21), device="cuda")
    x = torch.randn((T, 256), generator=new_gen(22), device="cuda").to(BF)
    step = lambda: layer(a, p, x, w, c.cache, c.batch, f, heads, c.prefix if shared else None)[0]  # noqa: E731
    step()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        held = step()
    for turn in range(4):
        x.copy_(torch.randn((T, 256), generator=new_gen(23 + turn), device="cuda"))
        c.lengths.copy_(ints([[200, 130, 64], [70, 200, 60], [64, 65, 66], [180, 100, 199]][turn]))
        keys, values = c.keys.clone(), c.values.clone()
        graph.replay()
        torch.cuda.synchronize()
        got = held.clone(), c.keys.clone(), c.values.clone()
        c.keys.copy_(keys)
        c.values.copy_(values)
        want = step()
        torch.cuda.synchronize()
        assert torch.equal(got[0], want) and torch.equal(got[1], c.keys) and torch.equal(got[2], c.values), turn


def test_two_graphs_and_two_streams_at_once(a):
    """Two captured calls replayed together on two streams, and eager ones on a third: no scratch is shared."""
    case("two graphs")
    calls = [Call(a, [(1, 3000), (1, 900)], 4, 2, 128, 16, BF, seed=24), Call(a, [(200, 900), (70, 500)], 4, 2, 128, 16, BF, seed=25),
             Call(a, [(1, 5000), (1, 70)], 4, 2, 128, 16, BF, seed=26, prefixes=[2000], starts=[0, 2])]
    run = lambda c, **k: a.attend_shared(c.q, c.cache, c.batch, c.prefix, **k) if c.prefixes else a.attend(c.q, c.cache, c.batch, **k)  # noqa: E731
    want = [run(c) for c in calls]
    graphs, outs, streams = [], [], [torch.cuda.Stream() for _ in range(3)]
    torch.cuda.synchronize()
    for c in calls[:2]:
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            outs.append(run(c))
        graphs.append(g)
    torch.cuda.synchronize()
    for _ in range(20):
        for g, s in zip(graphs, streams):
            with torch.cuda.stream(s):
                g.replay()
        got = run(calls[2], stream=streams[2])
    torch.cuda.synchronize()
    for y, right in zip(outs + [got], want):
        assert torch.equal(y, right)


@pytest.mark.parametrize("raw", [False, True], ids=["stream", "handle"])
def test_stream_argument_waits_for_what_the_stream_holds(a, raw):
    """The inputs get their values on the given stream, behind work that is still running when the calls are made."""
    case("stream order", raw)
    s = torch.cuda.Stream()
    stream = s.cuda_stream if raw else s
    c = Call(a, [(1, 300), (2, 90)], 4, 2, 64, 16, BF, seed=27, prefixes=[60], starts=[0, 2])
    old, new = torch.zeros_like(c.q), c.q.clone()
    f, at = torch.rand(32, generator=new_gen(28), device="cuda"), torch.arange(3, device="cuda").int()
    k = new[:, :2].contiguous()
    calls = {"attend": lambda x, **o: a.attend(x, c.cache, c.batch, **o),
             "shared": lambda x, **o: a.attend_shared(x, c.cache, c.batch, c.prefix, **o),
             "rotate": lambda x, **o: a.rotate_heads(x, at, f, **o),
             "append": lambda x, **o: a.append_heads(x, k, k, c.cache, c.batch, f, **o)}
    busy = torch.randn((4096, 4096), generator=new_gen(29), device="cuda")
    for name in ("attend", "shared", "rotate", "append"):
        call = calls[name]
        want = call(new)
        given, written = old.clone(), torch.cuda.Event()
        call(given)
        torch.cuda.synchronize()
        with torch.cuda.stream(s):
            for _ in range(50):  # tens of milliseconds
                torch.mm(busy, busy)
            given.copy_(new)
            written.record(s)
        got = call(given, stream=stream)
        assert not written.query(), name
        torch.cuda.synchronize()
        assert torch.equal(got, want), name


def test_same_bits_every_time(a):
    case("repeat")
    for requests, prefixes in (([(1, 5000)] * 3, []), ([(8, 900)] * 30, []), ([(700, 2000), (300, 300)], []), ([(1, 90)] * 50, [3001])):
        c = Call(a, requests, 10, 2, 128, 16, BF, seed=30, prefixes=prefixes, starts=[0, len(requests)])
        run = lambda: a.attend_shared(c.q, c.cache, c.batch, c.prefix) if prefixes else a.attend(c.q, c.cache, c.batch)  # noqa: E731
        one = run()
        for _ in range(5):
            assert torch.equal(run(), one)


GUARD = 1 << 16


def guarded(size):
    """`size` bytes between two guards, and whether those are as they were."""
    all_ = torch.full((2 * GUARD + size,), 0xa5, dtype=torch.uint8, device="cuda")
    return all_[GUARD:GUARD + size], lambda: bool((all_[:GUARD] == 0xa5).all()) and bool((all_[GUARD + size:] == 0xa5).all())


@TYPES
@pytest.mark.parametrize("layout", range(9))
def test_attend_stays_inside_its_scratch_and_output(a, layout, dtype):
    requests, prefixes, Hq, D = [([(1, 4000)], [], 4, 128), ([(1, 900)] * 60, [], 16, 64), ([(9, 700)] * 20, [], 4, 128), ([(16, 600)] * 9, [], 8, 256), ([(300, 900), (70, 70)], [], 4, 136),
                                 ([(2, 50)] * 30, [2000, 300], 4, 128), ([(150, 150), (1, 40)], [257], 4, 256), ([(200, 200 + 90 * b) for b in range(6)], [], 8, 128),
                                 ([(700, 700), (3, 2000)], [], 4, 72)][layout]
    case("scratch", layout, dtype)
    G = len(prefixes)
    c = Call(a, requests, Hq, 2, D, 16, dtype, seed=31, prefixes=prefixes, starts=[len(requests) * g // G for g in range(G + 1)] if G else None)
    lib = a.library()
    size = lib.hc_attend_work(c.T, Hq, 2, D, len(requests), G)
    assert size > 0
    work, untouched = guarded(size)
    out, kept = guarded(2 * c.q.numel())
    handle = torch.cuda.current_stream().cuda_stream
    for short in (1, 0):
        rest = (c.scale, 0.0, None, None, None, out.data_ptr(), Hq * D, D, work.data_ptr(), size - short, handle)
        if G:
            status = lib.hc_attend_shared(c.T, Hq, c.q.data_ptr(), Hq * D, D, c.cache._at, c.batch._at, c.prefix._at, *rest)
        else:
            status = lib.hc_attend(c.T, Hq, c.q.data_ptr(), Hq * D, D, c.cache._at, c.batch._at, *rest)
        assert (status == a.HC_OK) == (short == 0)
    assert untouched() and kept()
    c.check(out.view(dtype).view(c.q.shape), c.want())
