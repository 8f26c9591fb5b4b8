"""attend_shared and append_heads at the head shapes and numbers of requests that test_gpu_attention.py has for attend."""
import pytest
import torch

from test_gpu_attention import BF, HF, SHARED, TYPES, Call, a, case, check_turned, new_gen, ranges  # noqa: F401 (a: the fixture)

pytestmark = pytest.mark.gpu


@TYPES
@pytest.mark.parametrize("kind", [None, "window", "documents", "prefix", "any"])
@pytest.mark.parametrize("cap,bias", [(0.0, True), (20.0, False), (90.0, True)])
@pytest.mark.parametrize("layout,Hq,Hkv,D,page", [(4, 5, 1, 128, 16), (3, 4, 2, 256, 32), (5, 6, 3, 96, 16), (7, 4, 2, 136, 64), (5, 10, 2, 128, 16)])
def test_masks_cap_and_bias(a, layout, Hq, Hkv, D, page, cap, bias, kind, dtype):
    case("shared masks", layout, Hq, Hkv, D, page, cap, bias, kind, dtype)
    requests, prefixes, starts = SHARED[layout]
    c = Call(a, requests, Hq, Hkv, D, page, dtype, seed=61, prefixes=prefixes, starts=starts)
    first, last = ranges(c, kind) if kind else (None, None)
    slopes = torch.exp2(-torch.arange(1, Hq + 1, device="cuda") * 8.0 / Hq) if bias else None
    got = a.attend_shared(c.q, c.cache, c.batch, c.prefix, cap=cap, slopes=slopes, first=first, last=last)
    c.check(got, c.want(cap=cap, slopes=slopes, first=first, last=last))


MANY = {  # requests, prefixes, starts: more than 64 segments, tiles of several kinds
    "prompts": ([(150 + b, 200 + b) for b in range(9)] + [(1, 30)] * 70, [300, 129], [0, 9, 79]),
    "2000 of 40": ([(1, 1 + b % 30) for b in range(2000)], [50 + 3 * g for g in range(40)], [50 * g for g in range(41)]),
    "some without": ([(b % 4, 5 + b % 70) for b in range(300)], [400, 1, 77], [20, 100, 100, 290]),
}


@pytest.mark.parametrize("masked", [False, True])
@pytest.mark.parametrize("name", MANY)
@pytest.mark.parametrize("Hq,Hkv,D", [(2, 2, 64), (5, 1, 128), (2, 1, 256)])
def test_many_requests(a, name, Hq, Hkv, D, masked):
    case("shared many", name, Hq, Hkv, D, masked)
    requests, prefixes, starts = MANY[name]
    c = Call(a, requests, Hq, Hkv, D, 16, BF, seed=62, prefixes=prefixes, starts=starts)
    first, last = ranges(c, "any") if masked else (None, None)
    c.check(a.attend_shared(c.q, c.cache, c.batch, c.prefix, first=first, last=last), c.want(first=first, last=last))


@pytest.mark.parametrize("B,new", [(2048, lambda b: 1), (2048, lambda b: b % 3), (1500, lambda b: 1 + 9 * (b % 100 == 7)), (65, lambda b: 0 if b < 64 else 40)])
def test_append_to_many_requests(a, B, new):
    """The request of a token is looked for among all of them, empty ones too."""
    case("append many", B)
    c = Call(a, [(new(b), max(1, new(b)) + b % 40) for b in range(B)], 2, 2, 64, 16, HF, seed=63)
    gen = new_gen(64)
    q, k, v = (torch.randn((c.T, 2, 64), generator=gen, device="cuda").to(HF) for _ in range(3))
    f = torch.rand(32, generator=gen, device="cuda")
    got = a.append_heads(q, k, v, c.cache, c.batch, f)
    p = torch.cat([torch.arange(L - n, L) for n, L in c.requests]).cuda()
    b = torch.repeat_interleave(torch.arange(B), torch.tensor([n for n, _ in c.requests])).cuda()
    at = c.table[b, p // 16].long(), p % 16
    check_turned(got, q, p, f, None, 1e-6, False)
    check_turned(c.keys[at], k, p, f, None, 1e-6, False)
    assert torch.equal(c.values[at], v)
    none = a.append_heads(q[:, :0], k, v, c.cache, c.batch, f)
    assert none.shape == (c.T, 0, 64)
