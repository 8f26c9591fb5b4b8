"""Where the attention's numbers run out of digits.  Oracles in 64 bits; bounds
from the half step of a rounding (bf16 2^-8, fp16 2^-11, fp32 2^-24, relative)."""
import math

import pytest
import torch

from test_gpu_attention import BF, HF, NAN, TYPES, Call, a, case, ints, new_gen  # noqa: F401 (a: the fixture)

pytestmark = pytest.mark.gpu


class Far:
    """Requests whose tables lead, page after page, to the same few pages, so that their positions may be as far as one
    likes; of them, token t sees the last `window` up to its own."""

    def __init__(self, a, news, lengths, Hq, Hkv, D, page, dtype, window, prefix=0):
        gen = new_gen(sum(news) + D)
        self.page, self.Hq, self.Hkv, self.D, self.dtype, self.prefix = page, Hq, Hkv, D, dtype, prefix
        self.keys, self.values = (torch.randn((7, page, Hkv, D), generator=gen, device="cuda").to(dtype) for _ in range(2))
        width = lambda n: max(1, -(-n // page))  # noqa: E731
        self.table = (torch.arange(width(max(lengths)), device="cuda").int() * 3 % 7).repeat(len(news), 1).contiguous()
        self.cache = a.PagedCache(self.keys, self.values)
        off = [0]
        for n in news:
            off.append(off[-1] + n)
        self.batch = a.Batch(ints(off), ints(lengths), self.table)
        self.T = off[-1]
        p = torch.cat([torch.arange(L - n, L) for n, L in zip(news, lengths)]) + prefix
        self.p = p.cuda()
        self.first = (p - window + 1).clamp(min=0).int().cuda()
        self.prefix_table = (torch.arange(width(prefix), device="cuda").int() * 5 % 7)[None].contiguous()
        self.shared = a.SharedPrefix(ints([0, len(news)]), ints([prefix]), self.prefix_table) if prefix else None
        self.q = torch.randn((self.T, Hq, D), generator=gen, device="cuda").to(dtype)

    def want(self, slopes, last=None):
        """(results, bounds): attention over first <= j < last, in 64 bits."""
        out = torch.zeros((self.T, self.Hq, self.D), dtype=torch.float64, device="cuda")
        bound = out.clone()
        u = torch.finfo(self.dtype).eps / 2
        for t in range(self.T):
            j = torch.arange(int(self.first[t]), int(self.p[t]) + 1 if last is None else int(last[t]), device="cuda")
            own = (j - self.prefix).clamp(min=0)
            b = int((self.batch.offsets[1:] <= t).sum())
            at = torch.where(j < self.prefix, self.prefix_table[0, (j // self.page).clamp(max=self.prefix_table.shape[1] - 1)], self.table[b, own // self.page]).long()
            row = torch.where(j < self.prefix, j, own) % self.page
            k, v = (x[at, row].double().repeat_interleave(self.Hq // self.Hkv, 1) for x in (self.keys, self.values))
            q = self.q[t].double()
            z = (q * k).sum(-1).T * self.D ** -0.5
            size = (q.abs() * k.abs()).sum(-1).T * self.D ** -0.5
            far = slopes.double()[:, None] * (self.p[t] - j).abs()
            # scores: D steps of an fp32 sum (2^-23 each); scaling, bias, difference: 8 roundings of what they are made of
            e = (self.D + 8) * 2.0 ** -23 * size + 8 * 2.0 ** -23 * far
            z = z - far
            e = torch.where(z > z.amax(1, keepdim=True) - 40, e, 0.0).amax(1)
            w = torch.softmax(z, 1)
            y, mag = ((w[:, :, None] * x.permute(1, 0, 2)).sum(1) for x in (v, v.abs()))
            out[t] = y
            # numerators' rounding, their relative errors in sum and weights, the sums' order, the output's rounding
            bound[t] = (u + 2 * torch.expm1(e)[:, None] + (2 * len(j) + 32) * 2.0 ** -23) * mag + u * y.abs()
            if self.dtype == HF:
                bound[t] += 2.0 ** -25 * (1 + len(j) * float(self.values.abs().max()))
        return out, bound


@TYPES
@pytest.mark.parametrize("news,lengths,Hq,Hkv,D,page", [([1, 1], [2 ** 24 + 77, 2 ** 25 + 1001], 5, 1, 128, 65536), ([3, 2], [2 ** 26 + 5, 2 ** 24 + 3], 4, 2, 256, 65536),
                                                        ([20, 1], [2 ** 24 + 41, 60], 4, 2, 64, 4096), ([70], [2 ** 27 + 9], 8, 4, 128, 65536), ([20], [2 ** 24 + 1], 4, 1, 256, 65536)])
def test_distances_of_far_positions(a, news, lengths, Hq, Hkv, D, page, dtype):
    """Past 2^24, positions are no numbers of fp32, but their distances are."""
    case("far positions", news, lengths, Hq, Hkv, D, dtype)
    c = Far(a, news, lengths, Hq, Hkv, D, page, dtype, 100)
    slopes = torch.tensor([0.5, 1.0, 2.0, 0.25, 3.0, 0.75, 0.1, 1.5], device="cuda")[:Hq].contiguous()
    got = a.attend(c.q, c.cache, c.batch, slopes=slopes, first=c.first)
    want, bound = c.want(slopes)
    assert bool(((got.double() - want).abs() <= bound).all()), float(((got.double() - want).abs() / bound).max())
    last = torch.minimum(c.p + 30, torch.cat([torch.full((n,), L, device="cuda") for n, L in zip(news, lengths)])).int()  # later ones, too
    got = a.attend(c.q, c.cache, c.batch, slopes=slopes, first=c.first, last=last)
    want, bound = c.want(slopes, last)
    assert bool(((got.double() - want).abs() <= bound).all()), float(((got.double() - want).abs() / bound).max())


@TYPES
@pytest.mark.parametrize("D", [64, 128, 256])
def test_distances_of_far_positions_under_a_prefix(a, D, dtype):
    case("far positions under a prefix", D, dtype)
    c = Far(a, [1, 4, 30], [20, 40, 90], 4, 2, D, 65536, dtype, 120, prefix=2 ** 25 + 13)
    slopes = torch.tensor([0.5, 1.0, 0.05, 0.2], device="cuda")
    got = a.attend_shared(c.q, c.cache, c.batch, c.shared, slopes=slopes, first=c.first)
    want, bound = c.want(slopes)
    assert bool(((got.double() - want).abs() <= bound).all()), float(((got.double() - want).abs() / bound).max())


def alike(a, B, n, L, Hkv, D, dtype, scores, values):
    """B requests of n tokens that all see the same L positions, of these scores over ln 2 and these values: the smallest
    and the largest number of the results, and what all of them are."""
    keys, kept = torch.zeros((L // 16, 16, Hkv, D), dtype=dtype, device="cuda"), torch.zeros((L // 16, 16, Hkv, D), dtype=dtype, device="cuda")
    top = float(scores.abs().max())
    k = (scores / top).to(dtype)
    keys[..., 0] = k.view(-1, 16, 1).expand(-1, -1, Hkv)
    kept[:] = values.to(dtype).view(-1, 16, 1, 1)
    q = torch.zeros((B * n, Hkv, D), dtype=dtype, device="cuda")
    q[..., 0] = 1
    table = torch.arange(L // 16, device="cuda").int().repeat(B, 1).contiguous()
    batch = a.Batch(ints([n * b for b in range(B + 1)]), ints([L] * B), table)
    scale = top * math.log(2.0)
    got = a.attend(q, a.PagedCache(keys, kept), batch, scale=scale, last=ints([L] * (B * n)))
    z = torch.tensor(scale, dtype=torch.float32).double().item() * k.double()
    want = float(torch.softmax(z, 0) @ values.to(dtype).double())
    return (float(got.min()), float(got.max())), want


@TYPES
@pytest.mark.parametrize("top", [3e7, 1.7e9, 7e11, 1e30])
@pytest.mark.parametrize("B,n,Hkv,D", [(3, 1, 4, 64), (3, 1, 2, 256), (5, 20, 4, 64), (5, 20, 4, 128), (5, 40, 2, 256), (3, 300, 2, 128)])
def test_large_scores(a, B, n, Hkv, D, top, dtype):
    """Scores whose last bit is more than the exponential's range: the result is the largest one's value, or the mean of
    two that are equal, whatever comes before them."""
    case("large scores", B, n, Hkv, D, top, dtype)
    L = 512
    for sign in (1.0, -1.0):
        for at in ([0], [400], [100, 401]):
            scores = torch.linspace(-1.0, 0.96, L, device="cuda") * top if sign > 0 else torch.full((L,), -top, device="cuda")
            values = torch.randn(L, generator=new_gen(len(at)), device="cuda")
            scores[at] = top if sign > 0 else -0.96 * top
            got, want = alike(a, B, n, L, Hkv, D, dtype, scores, values)
            # (the weights are 1, or two of 1/2: the output's rounding)
            assert all(abs(x - want) <= (torch.finfo(dtype).eps / 2 + 2.0 ** -20) * abs(want) for x in got), (sign, at, got, want)


@pytest.mark.parametrize("B,n,Hkv,D", [(128, 1, 4, 64), (128, 1, 4, 128), (128, 1, 2, 256), (128, 20, 4, 64), (128, 20, 4, 128), (128, 40, 2, 256), (130, 300, 2, 128)])
def test_many_small_weights_under_a_large_one(a, B, n, Hkv, D):
    """8192 positions of 2^-25.5 of the largest weight each: numerators that fp16 would round to nothing next to one of 1.
    With the largest at 2^11 to 2^15, a numerator is off by up to 2^-36 of the largest, or by half a step."""
    case("small weights", B, n, Hkv, D)
    L = 8192
    for far in (25.5, 29.3):
        scores, values = torch.zeros(L, device="cuda"), torch.full((L,), 512.0, device="cuda")
        scores[0:128:32] = far  # (a position for each of the waves that may share a row)
        values[0:128:32] = 0.0
        got, want = alike(a, B, n, L, Hkv, D, HF, scores, values)
        u = 2.0 ** -11
        # scores: 8 roundings of `far` (fp32, over ln 2), which move a weight by ln 2 times that
        bound = (2 * u + 2 * 8 * 2.0 ** -23 * far + (2 * L + 32) * 2.0 ** -23) * want + 2.0 ** -36 * (L * 512.0)
        print(far, got, want, bound, flush=True)
        assert all(abs(x - want) <= bound for x in got)


@TYPES
@pytest.mark.parametrize("B,n,Hkv,D", [(128, 1, 4, 64), (128, 1, 2, 256), (128, 20, 4, 64), (128, 20, 4, 128), (130, 300, 2, 128)])
def test_large_values(a, B, n, Hkv, D, dtype):
    """Sums of values that are numbers of fp32, under scores that rise as they are read."""
    case("large values", B, n, Hkv, D, dtype)
    L = 512
    scores, values = torch.zeros(L, device="cuda"), torch.full((L,), 2.0 ** 118 if dtype == BF else 60000.0, device="cuda")
    for step in (3.9, 7.9):
        scores[256:] = step
        got, want = alike(a, B, n, L, Hkv, D, dtype, scores, values)
        print(step, got, want, flush=True)
        # numerators' rounding (twice: no two need be alike), sums' order, the output's rounding
        assert all(abs(x - want) <= (3 * torch.finfo(dtype).eps / 2 + (2 * L + 32) * 2.0 ** -23) * want for x in got)


@TYPES
@pytest.mark.parametrize("requests,Hq,Hkv,D", [([(1, 8), (1, 9), (1, 40)], 4, 4, 64), ([(1, 8), (2, 30), (1, 17), (1, 8)], 10, 2, 128), ([(1, 33)] * 40, 4, 2, 104),
                                               ([(1, 12), (4, 25)], 8, 2, 256), ([(8, 40), (5, 21)], 8, 2, 256)])
def test_few_rows_numerators_keep_their_digits(a, requests, Hq, Hkv, D, dtype):
    """Of few rows, numerators enter the second product in two pieces of the 16-bit type: what one rounding leaves (u of it)
    is rounded again, u^2 in all, in fp16 down to 2^-25 of 2^11."""
    case("digits", requests[0], Hq, Hkv, D, dtype)
    c = Call(a, requests, Hq, Hkv, D, 16, dtype, seed=51, sigma=0.05)
    got = a.attend(c.q, c.cache, c.batch)
    out, size, error = c.want()
    u, n = torch.finfo(dtype).eps / 2, max(L for _, L in requests)
    bound = (u * u + 2 * torch.expm1(error)[..., None] + (2 * n + 32) * 2.0 ** -23) * size + u * out.abs()
    if dtype == HF:
        bound += 2.0 ** -36 * n * 8 + 2.0 ** -25  # (values below 8; the output's own smallest step)
    assert float(torch.nan_to_num(c.values.float()).abs().max()) < 8
    assert bool(((got.double() - out).abs() <= bound).all()), float(((got.double() - out).abs() / bound).max())


@pytest.mark.parametrize("B,n,Hkv,D", [(128, 1, 4, 64), (3, 1, 2, 256), (128, 20, 4, 64), (3, 20, 4, 128), (130, 300, 2, 128)])
def test_large_values_of_no_weight(a, B, n, Hkv, D):
    """Values next to fp32's largest in sum, of weights that are nothing: they leave nothing."""
    case("large values of no weight", B, n, Hkv, D)
    L = 512
    scores, values = torch.zeros(L, device="cuda"), torch.ones(L, device="cuda")
    values[:256] = 2.0 ** 119
    scores[256:] = 1000.0
    got, want = alike(a, B, n, L, Hkv, D, BF, scores, values)
    # (the numerators are powers of two: the output's rounding, and what is left of 2^127)
    assert want == 1.0 and all(abs(x - want) <= 2.0 ** -8 + 2.0 ** -20 for x in got), got


@TYPES
@pytest.mark.parametrize("requests,prefixes,Hq,Hkv,D", [([(60, 300)], [], 4, 2, 64), ([(300, 3000)], [], 5, 1, 128), ([(40, 900)], [], 2, 1, 256), ([(3, 200), (1, 7)], [], 4, 1, 256),
                                                       ([(1, 40)] * 20, [500], 4, 2, 128), ([(9, 40), (30, 60)], [100], 2, 2, 64)])
def test_large_scores_of_others_change_no_bit(a, requests, prefixes, Hq, Hkv, D, dtype):
    """Tokens whose scores are large, infinite or no numbers share waves with tokens whose are not."""
    case("others", requests[0], prefixes, Hq, Hkv, D, dtype)
    c = Call(a, requests, Hq, Hkv, D, 16, dtype, seed=52, prefixes=prefixes, starts=[0, len(requests)], sigma=0.1)
    run = lambda q: a.attend_shared(q, c.cache, c.batch, c.prefix, scale=4.0) if prefixes else a.attend(q, c.cache, c.batch, scale=4.0)  # noqa: E731
    want = run(c.q)
    for t in {0, 1 % c.T, c.T // 2, c.T - 1}:
        for bad in (6e4, -6e4, math.inf, NAN):  # (scores of 2^21 and more, over ln 2)
            q = c.q.clone()
            q[t] = q[t].sign() * bad if math.isfinite(bad) else bad
            got = run(q)
            got[t] = want[t]
            assert torch.equal(got, want), (t, bad)
    # a key that only the last token of the last request sees
    b, (n, L) = len(requests) - 1, requests[-1]
    at = int(c.table[b, (L - 1) // 16]), (L - 1) % 16
    signs = c.q[-1, ::Hq // Hkv].sign()  # (all products of the last token's first heads of one sign)
    for bad in (6e4, -6e4, math.inf, -math.inf):
        kept = c.keys[at].clone()
        c.keys[at] = bad * signs
        got = run(c.q)
        c.keys[at] = kept
        got[-1] = want[-1]
        assert torch.equal(got, want), bad
