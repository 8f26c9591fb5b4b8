"""The attention's C ABI and binding on the host: what the header declares is
what the library exports, and bad arguments are refused before any HIP call."""
import ctypes
import math
import os
import random
import re
import subprocess

import pytest
import torch

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
HEADER = os.path.join(ROOT, "include", "hc_attn.h")
GOOD = 0x10000  # never dereferenced: the checks reject first
NO_GPU = not (os.path.exists("/dev/kfd") and os.access("/dev/kfd", os.R_OK))
ARG, ALIGN, DEVICE, SIZE = 1, 2, 3, 6


@pytest.fixture(scope="module")
def a():
    from hyper_connection_residual_amd import attention
    if not os.path.exists(attention.LIB_PATH):
        from hyper_connection_residual_amd import build
        build.build_attention()
    attention.library()
    return attention


def test_library_exports_what_the_header_declares(a):
    declared = re.findall(r"HC_API\s+[\w\s\*]+?\b(hc_\w+)\s*\(", open(HEADER).read())
    assert set(declared) == set(a.SIGNATURES) and len(declared) == len(set(declared))
    out = subprocess.run(["nm", "-D", "--defined-only", a.LIB_PATH], capture_output=True, text=True, check=True).stdout
    assert {l.split()[-1] for l in out.splitlines() if " T " in l} == set(declared)


def test_binding_constants_and_structures_are_the_headers(a):
    text = open(HEADER).read()
    for name in ("HC_MAX_HEAD", "HC_MAX_REQUESTS", "HC_MAX_ROWS", "HC_MIN_PAGE", "HC_MAX_PAGE"):
        assert int(re.search(r"#define %s (\d+)" % name, text).group(1)) == getattr(a, name)
    for name in ("hc_cache", "hc_batch", "hc_prefix"):
        body = re.sub(r"/\*.*?\*/", "", re.search(r"struct %s \{(.*?)\} %s;" % (name, name), text, re.S).group(1), flags=re.S)
        fields = [f.strip(" *") for line in body.split(";") if line.strip() for f in re.sub(r"^\s*(const\s+)?\w+", "", line.strip()).split(",")]
        assert fields == [n for n, _ in getattr(a, name)._fields_]


def cache(a, **change):
    c = dict(keys=GOOD, values=GOOD, pages=9, page_size=16, heads=2, dim=64, key_page=2048, key_row=128, key_head=64, value_page=2048,
             value_row=128, value_head=64, type=0)
    assert set(change) <= set(c)
    c.update(change)
    return a.hc_cache(*c.values())


def batch(a, **change):
    b = dict(requests=3, offsets=GOOD, lengths=GOOD, table=GOOD, width=5, table_row=5)
    assert set(change) <= set(b)
    b.update(change)
    return a.hc_batch(*b.values())


def prefix(a, **change):
    p = dict(groups=2, starts=GOOD, lengths=GOOD, table=GOOD, width=5, table_row=5)
    assert set(change) <= set(p)
    p.update(change)
    return a.hc_prefix(*p.values())


def split(change, of):
    """The changes that belong to a description, and the rest."""
    return {k[len(of) + 1:]: v for k, v in change.items() if k.startswith(of + ".")}, {k: v for k, v in change.items() if not k.startswith(of + ".")}


def call(a, name, **change):
    c, change = split(change, "cache")
    b, change = split(change, "batch")
    p, change = split(change, "prefix")
    c, b, p = cache(a, **c), batch(a, **b), prefix(a, **p)
    if name == "hc_rotate_heads":
        args = dict(T=4, heads=8, dim=64, type=0, x=GOOD, x_row=512, x_head=64, positions=GOOD, frequencies=GOOD, rotated=64, interleaved=0,
                    weight=GOOD, eps=1e-6, out=GOOD, out_row=512, out_head=64, stream=0)
    elif name == "hc_append_heads":
        args = dict(T=4, q_heads=8, q=GOOD, q_row=512, q_head=64, k=GOOD, k_row=128, k_head=64, v=GOOD, v_row=128, v_head=64,
                    cache=ctypes.addressof(c), batch=ctypes.addressof(b), positions=GOOD, frequencies=GOOD, rotated=64, interleaved=0,
                    q_weight=GOOD, k_weight=GOOD, eps=1e-6, out=GOOD, out_row=512, out_head=64, stream=0)
    else:
        args = dict(T=4, q_heads=8, q=GOOD, q_row=512, q_head=64, cache=ctypes.addressof(c), batch=ctypes.addressof(b))
        if name == "hc_attend_shared":
            args["prefix"] = ctypes.addressof(p)
        args.update(scale=0.125, cap=0.0, slopes=GOOD, first=GOOD, last=GOOD, out=GOOD, out_row=512, out_head=64, work=GOOD,
                    work_bytes=1 << 40, stream=0)
    assert set(change) <= set(args)
    args.update(change)
    return getattr(a.library(), name)(*args.values())


NAN, INF = math.nan, math.inf
CACHE_ARG = [dict(cache=None)] + [{"cache." + k: v} for k, v in (
    ("keys", None), ("values", None), ("pages", 0), ("page_size", 0), ("heads", 0), ("dim", 0), ("type", 2), ("type", -1), ("key_row", 56),
    ("value_row", 56), ("key_head", 32), ("value_head", 56), ("key_page", -8), ("value_page", -2048))]
CACHE_SIZE = [{"cache." + k: v} for k, v in (
    ("page_size", 8), ("page_size", 48), ("page_size", 1 << 17), ("pages", 1 << 31), ("key_row", 132), ("value_head", 68), ("key_page", 2052),
    ("key_row", 1 << 23), ("value_head", 1 << 23), ("key_page", (1 << 31) - 65536), ("value_page", 1 << 31))] + [{"cache.dim": 60}, {"cache.dim": 264, "cache.key_row": 528, "cache.value_row": 528, "cache.key_head": 264, "cache.value_head": 264}]
CACHE_ALIGN = [{"cache.keys": GOOD + 8}, {"cache.values": GOOD + 2}]
BATCH_ARG = [dict(batch=None)] + [{"batch." + k: v} for k, v in (
    ("requests", 0), ("offsets", None), ("lengths", None), ("table", None), ("width", -1), ("table_row", 4))]
BATCH_SIZE = [{"batch.requests": 2049}, {"batch.width": 1 << 31, "batch.table_row": 1 << 31}]
BATCH_ALIGN = [{"batch.offsets": GOOD + 2}, {"batch.lengths": GOOD + 1}, {"batch.table": GOOD + 2}]
ATTEND_ARG = CACHE_ARG + BATCH_ARG + [
    dict(T=0), dict(T=-4), dict(q_heads=0), dict(q_heads=7), dict(q=None), dict(out=None), dict(work=None), dict(cap=-1.0), dict(cap=NAN), dict(cap=INF),
    dict(scale=2e30), dict(scale=-2e30), dict(cap=2e30),
    dict(scale=NAN), dict(scale=INF), dict(q_row=56), dict(q_head=56), dict(out_row=0), dict(out_head=32)]
ATTEND_SIZE = CACHE_SIZE + BATCH_SIZE + [
    dict(q_row=516), dict(q_head=68), dict(out_row=516), dict(out_head=66), dict(work_bytes=1000), dict(work_bytes=-1), dict(T=1 << 16, q_heads=16), dict(T=(1 << 18) + 1, q_heads=2),
    dict(T=1 << 40), {"batch.width": 1 << 28, "batch.table_row": 1 << 28}, {"T": 16000, "batch.width": 1 << 24, "batch.table_row": 1 << 24}]
ATTEND_ALIGN = CACHE_ALIGN + BATCH_ALIGN + [dict(q=GOOD + 8), dict(out=GOOD + 2), dict(work=GOOD + 8), dict(slopes=GOOD + 2), dict(first=GOOD + 1),
                                            dict(last=GOOD + 2)]
REFUSED = [
    ("hc_rotate_heads", ARG, [dict(T=0), dict(heads=0), dict(dim=0), dict(type=2), dict(x=None), dict(out=None), dict(positions=None), dict(rotated=0),
                              dict(rotated=72), dict(eps=-1.0), dict(eps=NAN), dict(x_row=56), dict(x_head=56), dict(out_row=8), dict(out_head=0)]),
    ("hc_rotate_heads", SIZE, [dict(T=1 << 31), dict(heads=65537), dict(dim=264, x_head=264, x_row=2112, out_head=264, out_row=2112), dict(dim=60, rotated=56), dict(rotated=12),
                               dict(x_row=516), dict(out_head=68), dict(T=(1 << 31) - 65536, heads=65536)]),
    ("hc_rotate_heads", ALIGN, [dict(x=GOOD + 8), dict(out=GOOD + 2), dict(positions=GOOD + 2), dict(frequencies=GOOD + 2), dict(weight=GOOD + 1)]),
    ("hc_append_heads", ARG, CACHE_ARG + BATCH_ARG + [
        dict(T=0), dict(q_heads=-1), dict(q=None), dict(k=None), dict(v=None), dict(out=None), dict(rotated=0), dict(rotated=72), dict(eps=-1.0), dict(q_row=8),
        dict(k_head=8), dict(v_row=56), dict(out_head=56)]),
    ("hc_append_heads", SIZE, CACHE_SIZE + BATCH_SIZE + [dict(T=1 << 31), dict(q_heads=65537), dict(rotated=12), dict(q_row=516), dict(k_row=132), dict(v_head=68),
                                                        dict(T=(1 << 31) - 65536, q_heads=65536)]),
    ("hc_append_heads", ALIGN, CACHE_ALIGN + BATCH_ALIGN + [dict(q=GOOD + 8), dict(k=GOOD + 2), dict(v=GOOD + 4), dict(out=GOOD + 8), dict(positions=GOOD + 2),
                                                            dict(frequencies=GOOD + 2), dict(q_weight=GOOD + 2), dict(k_weight=GOOD + 2)]),
    ("hc_attend", ARG, ATTEND_ARG),
    ("hc_attend", SIZE, ATTEND_SIZE),
    ("hc_attend", ALIGN, ATTEND_ALIGN),
    ("hc_attend_shared", ARG, ATTEND_ARG + [dict(prefix=None)] + [{"prefix." + k: v} for k, v in (
        ("groups", 0), ("starts", None), ("lengths", None), ("table", None), ("width", -1), ("table_row", 4))]),
    ("hc_attend_shared", SIZE, ATTEND_SIZE + [{"prefix.groups": 2049}, {"prefix.width": 1 << 28, "prefix.table_row": 1 << 28}]),
    ("hc_attend_shared", ALIGN, ATTEND_ALIGN + [{"prefix.starts": GOOD + 2}, {"prefix.lengths": GOOD + 1}, {"prefix.table": GOOD + 3}]),
]


@pytest.mark.parametrize("name,status,changes", REFUSED, ids=["%s-%d" % r[:2] for r in REFUSED])
def test_refusals_come_before_any_launch(a, name, status, changes):
    for change in changes:
        assert call(a, name, **change) == status, change


@pytest.mark.skipif(not NO_GPU, reason="a GPU is present; this checks the no-device error path")
def test_no_device_is_an_error_not_a_fallback(a):
    for name in ("hc_rotate_heads", "hc_append_heads", "hc_attend", "hc_attend_shared"):
        assert call(a, name) == DEVICE
    # what may be absent
    assert call(a, "hc_rotate_heads", positions=None, frequencies=None, weight=None, rotated=0) == DEVICE
    assert call(a, "hc_append_heads", q_heads=0, q=None, out=None, positions=None, frequencies=None, q_weight=None, k_weight=None) == DEVICE
    for name in ("hc_attend", "hc_attend_shared"):
        assert call(a, name, slopes=None, first=None, last=None) == DEVICE
        assert call(a, name, **{"batch.width": 0, "batch.table": None}) == DEVICE
    # strides of a dimension of one
    assert call(a, "hc_attend", q_heads=1, q_head=8, out_head=8, **{"cache.heads": 1, "cache.key_head": 8, "cache.value_head": 8, "cache.pages": 1,
                                                                 "cache.key_page": 0}) == DEVICE


def test_work_sizes(a):
    lib, rng = a.library(), random.Random(3)
    spread = lambda low, high: round(math.exp(rng.uniform(math.log(low), math.log(high))))  # noqa: E731
    assert lib.hc_attend_work(0, 4, 4, 64, 1, 0) == 0
    for bad in (dict(Hq=6), dict(D=60), dict(D=264), dict(B=2049), dict(B=0), dict(G=2049), dict(G=-1), dict(T=1 << 19)):
        v = dict(T=4, Hq=4, Hkv=4, D=64, B=2, G=0)
        v.update(bad)
        if bad.get("Hq"):
            v["Hkv"] = 4
        assert lib.hc_attend_work(*v.values()) == 0, bad
    for _ in range(3000):
        Hkv, g, D, B = spread(1, 32), spread(1, 16), 8 * rng.randint(1, 32), spread(1, 2048)
        T = spread(1, (1 << 18) // g)
        own, shared = lib.hc_attend_work(T, Hkv * g, Hkv, D, B, 0), lib.hc_attend_work(T, Hkv * g, Hkv, D, B, rng.randint(1, B))
        assert 0 < own < 160 << 20 and own < shared <= (160 << 20) + 2 * T * Hkv * g * (4 * 256 + 8)
        # the call takes exactly that much (refused for its size with a byte less, else for the device or not at all)
        if NO_GPU and D == 64:
            here = dict(T=T, q_heads=2 * g, work_bytes=lib.hc_attend_work(T, 2 * g, 2, 64, 3, 0))
            here.update(q_row=128 * g, out_row=128 * g)
            assert call(a, "hc_attend", **here) == DEVICE
            here["work_bytes"] -= 1
            assert call(a, "hc_attend", **here) == SIZE


def test_status_strings(a):
    texts = [a.hc_attn_status_string(s) for s in (0, ARG, ALIGN, DEVICE, 5, SIZE)]
    assert len(set(texts)) == 6 and all(texts) and "unknown status" not in texts
    assert a.hc_attn_status_string(99) == "unknown status"


def test_names_of_the_package():
    import hyper_connection_residual_amd as h
    from hyper_connection_residual_amd import attention
    for name in ("PagedCache", "Batch", "SharedPrefix", "rotate_heads", "append_heads", "attend", "attend_shared", "AttentionError"):
        assert name in h.__all__ and getattr(h, name) is getattr(attention, name)


B16, I32 = torch.bfloat16, torch.int32


def things(a):
    """A cache, batch and prefix on the CPU are refused, so their tensors stand in for them."""
    return torch.zeros((9, 16, 2, 64), dtype=B16), torch.zeros(4, dtype=I32), torch.zeros(3, dtype=I32), torch.zeros((3, 5), dtype=I32)


def test_descriptions_refuse_wrong_tensors(a):
    kv, off, lens, table = things(a)
    for make in (lambda: a.PagedCache(kv.float(), kv.float()), lambda: a.PagedCache(kv, kv.half()), lambda: a.PagedCache(None, kv), lambda: a.PagedCache(kv, [1]),
                 lambda: a.Batch(off.long(), lens, table), lambda: a.Batch(off, lens.float(), table), lambda: a.Batch(off, lens, table.long()),
                 lambda: a.Batch([0], lens, table), lambda: a.Batch(off, lens, None),
                 lambda: a.SharedPrefix(off.long(), lens, table), lambda: a.SharedPrefix(off, None, table), lambda: a.SharedPrefix(off, lens, 3)):
        with pytest.raises(TypeError):
            make()
    for make in (lambda: a.PagedCache(kv[0], kv[0]), lambda: a.PagedCache(kv, kv[:8]), lambda: a.PagedCache(kv[:, :8], kv[:, :8]),
                 lambda: a.PagedCache(kv[..., :60], kv[..., :60]), lambda: a.PagedCache(kv[:0], kv[:0]), lambda: a.PagedCache(kv.transpose(2, 3), kv.transpose(2, 3)),
                 lambda: a.PagedCache(kv.expand(9, 16, 2, 64)[:, :1].expand(9, 16, 2, 64), kv), lambda: a.PagedCache(kv[:, :, :1].expand(9, 16, 2, 64), kv),
                 lambda: a.PagedCache(torch.zeros((9, 16, 2, 68), dtype=B16)[..., :64], kv), lambda: a.PagedCache(torch.zeros((2, 24, 1, 64), dtype=B16), torch.zeros((2, 24, 1, 64), dtype=B16)),
                 lambda: a.PagedCache(torch.zeros((2, 16, 1, 264), dtype=B16), torch.zeros((2, 16, 1, 264), dtype=B16)),
                 lambda: a.PagedCache(*[torch.empty((2, 16, 2, 64), dtype=B16, device="meta").as_strided((2, 16, 2, 64), ((1 << 31) - 65536, 128, 64, 1))] * 2),
                 lambda: a.Batch(off[:3], lens, table), lambda: a.Batch(off, lens, table[:2]), lambda: a.Batch(off, lens, table[0]),
                 lambda: a.Batch(off[:1], lens[:0], table[:0]), lambda: a.Batch(off, lens, table.t().contiguous().t()),
                 lambda: a.Batch(torch.zeros(2050, dtype=I32), torch.zeros(2049, dtype=I32), torch.zeros((2049, 1), dtype=I32)),
                 lambda: a.SharedPrefix(off[:3], lens, table), lambda: a.SharedPrefix(off[:1], lens[:0], table[:0]), lambda: a.SharedPrefix(off, lens, table[:1])):
        with pytest.raises(ValueError):
            make()
    for make in (lambda: a.PagedCache(kv, kv), lambda: a.Batch(off, lens, table), lambda: a.SharedPrefix(off, lens, table),
                 lambda: a.Batch(off, lens, torch.zeros((3, 9), dtype=I32)[:, 2:7]), lambda: a.Batch(off, lens, table[:, :0]),
                 lambda: a.PagedCache(kv.transpose(1, 2).contiguous().transpose(1, 2), kv)):
        with pytest.raises(ValueError, match="GPU"):
            make()


@pytest.fixture
def made(a, monkeypatch):
    """Descriptions whose tensors lie on the CPU, for the checks of the calls."""
    monkeypatch.setattr(a, "_place", lambda *t: None)
    kv, off, lens, table = things(a)
    made = a.PagedCache(kv, kv), a.Batch(off, lens, table), a.SharedPrefix(off, lens, table)
    monkeypatch.undo()
    return made


def test_calls_refuse_wrong_arguments(a, made):
    cache, batch, prefix = made
    q, k, f, p = torch.zeros((4, 8, 64), dtype=B16), torch.zeros((4, 2, 64), dtype=B16), torch.zeros(32), torch.zeros(4, dtype=I32)
    w = torch.ones(64)
    for run in (lambda: a.rotate_heads(q.float()), lambda: a.rotate_heads(None), lambda: a.rotate_heads(q, p.long(), f), lambda: a.rotate_heads(q, p, f.double()),
                lambda: a.rotate_heads(q, p, f, weight=w.half()), lambda: a.rotate_heads(q, p, f, out=q.half()), lambda: a.rotate_heads(q, p, [1.0]),
                lambda: a.append_heads(q, k.half(), k, cache, batch), lambda: a.append_heads(q, k, k, None, batch), lambda: a.append_heads(q, k, k, cache, cache),
                lambda: a.append_heads(q.half(), k, k, cache, batch) if False else a.append_heads(q.float(), k, k, cache, batch),
                lambda: a.append_heads(q, k, k, cache, batch, f, positions=p.float()), lambda: a.append_heads(q, k, k, cache, batch, q_weight=w.double()),
                lambda: a.attend(q.half(), cache, batch), lambda: a.attend(q, batch, batch), lambda: a.attend(q, cache, None), lambda: a.attend(q, cache, batch, slopes=torch.zeros(8, dtype=B16)),
                lambda: a.attend(q, cache, batch, first=p.long()), lambda: a.attend(q, cache, batch, last=p.float()), lambda: a.attend(q, cache, batch, out=q.float()),
                lambda: a.attend_shared(q, cache, batch, None), lambda: a.attend_shared(q, cache, batch, batch)):
        with pytest.raises(TypeError):
            run()
    wide = torch.zeros((4, 8, 68), dtype=B16)
    for run in (lambda: a.rotate_heads(q[0]), lambda: a.rotate_heads(q[..., :60]), lambda: a.rotate_heads(wide[..., :64]), lambda: a.rotate_heads(q.transpose(1, 2)),
                lambda: a.rotate_heads(q[:, :1].expand(4, 8, 64)), lambda: a.rotate_heads(q[:1].expand(4, 8, 64)), lambda: a.rotate_heads(q, None, f),
                lambda: a.rotate_heads(q, p[:3], f), lambda: a.rotate_heads(q, p, torch.zeros(36)), lambda: a.rotate_heads(q, p, torch.zeros(6)), lambda: a.rotate_heads(q, p, torch.zeros(0)),
                lambda: a.rotate_heads(q, p, f, weight=w[:32]), lambda: a.rotate_heads(q, p, f, eps=-1.0), lambda: a.rotate_heads(q, p, f, eps=math.nan), lambda: a.rotate_heads(q, out=q[:3]),
                lambda: a.append_heads(q, k[:3], k, cache, batch), lambda: a.append_heads(q, k, q, cache, batch), lambda: a.append_heads(q[:3], k, k, cache, batch),
                lambda: a.append_heads(None, k, k, cache, batch, out=q), lambda: a.append_heads(q, k, k, cache, batch, f, positions=p[:2]), lambda: a.append_heads(q, k, k, cache, batch, k_weight=w[:8]),
                lambda: a.attend(q[:, :7], cache, batch), lambda: a.attend(q[..., :56], cache, batch), lambda: a.attend(q, cache, batch, cap=-1.0), lambda: a.attend(q, cache, batch, cap=1e31), lambda: a.attend(q, cache, batch, scale=-1e31), lambda: a.attend(q, cache, batch, scale=math.inf),
                lambda: a.attend(q, cache, batch, slopes=torch.zeros(7)), lambda: a.attend(q, cache, batch, first=p[:3]), lambda: a.attend(q, cache, batch, out=q[:2]), lambda: a.attend(q, cache, batch, out=q),
                lambda: a.attend(torch.zeros((1 << 17, 6, 64), dtype=B16), cache, batch)):
        with pytest.raises(ValueError):
            run()


def test_calls_refuse_cpu_tensors(a, made):
    cache, batch, prefix = made
    q, k, f, p = torch.zeros((4, 8, 64), dtype=B16), torch.zeros((4, 2, 64), dtype=B16), torch.zeros(32), torch.zeros(4, dtype=I32)
    for run in (lambda: a.rotate_heads(q, p, f), lambda: a.append_heads(q, k, k, cache, batch, f), lambda: a.attend(q, cache, batch), lambda: a.attend_shared(q, cache, batch, prefix),
                lambda: a.rotate_heads(q[:, :, :8]), lambda: a.append_heads(None, k, k, cache, batch)):
        with pytest.raises(ValueError, match="GPU"):
            run()
