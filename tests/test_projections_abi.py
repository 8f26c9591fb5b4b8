"""The projections' C ABI and binding on the host: what the header declares is
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
HEADER = os.path.join(ROOT, "include", "hc_proj.h")
GOOD = 0x10000  # never dereferenced: the checks reject first
NO_GPU = not (os.path.exists("/dev/kfd") and os.access("/dev/kfd", os.R_OK))


@pytest.fixture(scope="module")
def p():
    from hyper_connection_residual_amd import projections
    if not os.path.exists(projections.LIB_PATH):
        from hyper_connection_residual_amd import build
        build.build_projections()
    projections.library()
    return projections


def test_library_exports_what_the_header_declares(p):
    declared = re.findall(r"HC_API\s+[\w\s\*]+?\b(hc_\w+)\s*\(", open(HEADER).read())
    assert set(declared) == set(p.SIGNATURES) and len(declared) == len(set(declared))
    out = subprocess.run(["nm", "-D", "--defined-only", p.LIB_PATH], capture_output=True, text=True, check=True).stdout
    assert {l.split()[-1] for l in out.splitlines() if " T " in l} == set(declared)


def test_binding_constants_are_the_headers(p):
    text = open(HEADER).read()
    for name in ("HC_BF16", "HC_FP16", "HC_FP32", "HC_MAX_RANK", "HC_MAX_EXPERTS", "HC_MAX_TOPK"):
        assert int(re.search(r"#define %s (\d+)" % name, text).group(1)) == getattr(p, name)


def project_args(**change):
    a = dict(T=4, K=64, N=32, type=0, x=GOOD, ldx=64, W=GOOD, adapter=GOOD, adapters=2, rank=8, A=GOOD, B=GOOD,
             scale=GOOD, out=GOOD, ldo=32, out_type=0, work=GOOD, work_bytes=1 << 30, stream=0)
    assert set(change) <= set(a)
    a.update(change)
    return list(a.values())


def expert_args(**change):
    a = dict(R=4, K=64, N=32, E=2, type=0, x=GOOD, x_rows=4, ldx=64, rows=GOOD, W=GOOD, offsets=GOOD, gate=0, out=GOOD,
             ldo=32, out_type=0, stream=0)
    assert set(change) <= set(a)
    a.update(change)
    return list(a.values())


def route_args(**change):
    a = dict(T=4, E=8, k=2, logits=GOOD, ldl=8, type=2, renorm=1, ids=GOOD, weights=GOOD, offsets=GOOD, rows=GOOD,
             pos=GOOD, work=GOOD, work_bytes=1 << 30, stream=0)
    assert set(change) <= set(a)
    a.update(change)
    return list(a.values())


def combine_args(**change):
    a = dict(T=4, k=2, C=32, y=GOOD, y_rows=8, ldy=32, type=0, pos=GOOD, weights=GOOD, out=GOOD, ldo=32, out_type=2,
             stream=0)
    assert set(change) <= set(a)
    a.update(change)
    return list(a.values())


ARG, ALIGN, DEVICE, SIZE = 1, 2, 3, 6
REFUSED = [
    ("hc_project", project_args, ARG,
     [dict(T=0), dict(T=-3), dict(K=0), dict(N=0), dict(x=None), dict(W=None), dict(out=None), dict(type=2), dict(type=3),
      dict(type=-1), dict(out_type=1), dict(out_type=3), dict(ldx=56), dict(ldo=31), dict(A=None), dict(B=None),
      dict(rank=0), dict(adapters=-1), dict(work=None)]),
    ("hc_project", project_args, SIZE,
     [dict(K=60, ldx=64), dict(ldx=68), dict(rank=12), dict(rank=136), dict(work_bytes=16), dict(T=1 << 31),
      dict(N=1 << 31, ldo=1 << 31), dict(work_bytes=-1)]),
    ("hc_project", project_args, ALIGN,
     [dict(x=GOOD + 8), dict(W=GOOD + 2), dict(A=GOOD + 8), dict(B=GOOD + 8), dict(work=GOOD + 4), dict(out=GOOD + 1),
      dict(out_type=2, out=GOOD + 2), dict(adapter=GOOD + 2), dict(scale=GOOD + 2)]),
    ("hc_expert_project", expert_args, ARG,
     [dict(R=0), dict(K=0), dict(N=-1), dict(E=0), dict(x=None), dict(W=None), dict(offsets=None), dict(out=None),
      dict(type=2), dict(out_type=1), dict(ldx=8), dict(ldo=16), dict(x_rows=0), dict(rows=None, x_rows=3)]),
    ("hc_expert_project", expert_args, SIZE, [dict(K=68, ldx=72), dict(ldx=66), dict(R=1 << 31), dict(E=1 << 31)]),
    ("hc_expert_project", expert_args, ALIGN,
     [dict(x=GOOD + 8), dict(W=GOOD + 8), dict(offsets=GOOD + 2), dict(rows=GOOD + 1), dict(out=GOOD + 1)]),
    ("hc_route", route_args, ARG,
     [dict(T=0), dict(E=0), dict(k=0), dict(k=9), dict(logits=None), dict(ids=None), dict(weights=None),
      dict(offsets=None), dict(rows=None), dict(pos=None), dict(type=3), dict(ldl=7), dict(T=4096, work=None)]),
    ("hc_route", route_args, SIZE,
     [dict(E=513, ldl=513), dict(E=64, ldl=64, k=33), dict(T=1 << 31), dict(T=1 << 30), dict(T=4096, work_bytes=0)]),
    ("hc_route", route_args, ALIGN,
     [dict(logits=GOOD + 2), dict(ids=GOOD + 2), dict(weights=GOOD + 2), dict(offsets=GOOD + 2), dict(rows=GOOD + 2),
      dict(pos=GOOD + 2), dict(T=4096, work=GOOD + 8)]),
    ("hc_expert_combine", combine_args, ARG,
     [dict(T=0), dict(k=0), dict(C=0), dict(y_rows=0), dict(y=None), dict(pos=None), dict(weights=None), dict(out=None),
      dict(type=3), dict(out_type=-1), dict(ldy=31), dict(ldo=31)]),
    ("hc_expert_combine", combine_args, SIZE, [dict(T=1 << 31), dict(k=513), dict(T=1 << 22, C=1 << 22, ldy=1 << 22, ldo=1 << 22)]),
    ("hc_expert_combine", combine_args, ALIGN,
     [dict(y=GOOD + 1), dict(out=GOOD + 2), dict(pos=GOOD + 2), dict(weights=GOOD + 2)]),
]


@pytest.mark.parametrize("name,args,status,changes", REFUSED, ids=["%s-%d" % (r[0], r[2]) for r in REFUSED])
def test_refusals_come_before_any_launch(p, name, args, status, changes):
    fn = getattr(p.library(), name)
    for change in changes:
        assert fn(*args(**change)) == status, change


@pytest.mark.skipif(not NO_GPU, reason="a GPU is present; this checks the no-device error path")
def test_no_device_is_an_error_not_a_fallback(p):
    lib = p.library()
    for name, args in (("hc_project", project_args), ("hc_expert_project", expert_args), ("hc_route", route_args),
                       ("hc_expert_combine", combine_args)):
        assert getattr(lib, name)(*args()) == DEVICE
    # without adapters A, B, rank and (where no scratch is needed) work do not matter
    assert lib.hc_project(*project_args(adapter=None, A=None, B=None, rank=0, scale=None, work=None, work_bytes=0)) == DEVICE


def test_work_sizes(p):
    lib = p.library()
    assert lib.hc_project_work(1, 2560, 2560, 0) == 0
    assert lib.hc_project_work(1, 2560, 2560, 16) == 0
    assert lib.hc_project_work(2, 2560, 2560, 16) >= 4 * 2 * 16
    assert lib.hc_project_work(8192, 2560, 10240, 16) >= 4 * 8192 * 16
    assert lib.hc_project_work(0, 0, 0, 0) == 0
    assert lib.hc_route_work(8, 64, 8) == 0
    assert lib.hc_route_work(32768, 128, 8) > 0


def test_status_strings(p):
    texts = [p.hc_proj_status_string(s) for s in (0, ARG, ALIGN, DEVICE, 5, SIZE)]
    assert len(set(texts)) == 6 and all(texts) and "unknown status" not in texts
    assert p.hc_proj_status_string(99) == "unknown status"


def test_names_of_the_package():
    import hyper_connection_residual_amd as h
    from hyper_connection_residual_amd import projections
    for name in ("project", "route", "expert_project", "expert_combine", "ProjectionError"):
        assert name in h.__all__ and getattr(h, name) is getattr(projections, name)


def test_binding_refuses_wrong_types_and_shapes(p):
    b = torch.bfloat16
    x, W = torch.zeros((4, 64), dtype=b), torch.zeros((32, 64), dtype=b)
    ad = torch.zeros(4, dtype=torch.int32)
    A, B = torch.zeros((2, 8, 64), dtype=b), torch.zeros((2, 32, 8), dtype=b)
    off = torch.zeros(3, dtype=torch.int32)
    for call in (lambda: p.project(x.float(), W), lambda: p.project(x, W.half()), lambda: p.project(x, W, ad.long(), A, B),
                 lambda: p.project(x, W, ad, A, B.half()), lambda: p.project(x, W, out_dtype=torch.float16),
                 lambda: p.project(x, W, ad, A, B, scale=torch.zeros(2, dtype=torch.float64)),
                 lambda: p.project([1], W), lambda: p.project(x, None),
                 lambda: p.project(x, W, out=torch.empty((4, 32)), out_dtype=b),
                 lambda: p.expert_project(x.double(), W[None], off[:2]), lambda: p.expert_project(x, W[None], off[:2].long()),
                 lambda: p.route(torch.zeros((4, 8), dtype=torch.float64), 2),
                 lambda: p.expert_combine(x, ad.view(2, 2), torch.zeros((2, 2), dtype=b))):
        with pytest.raises(TypeError):
            call()
    for call in (lambda: p.project(x, W[:, :56]), lambda: p.project(x.t(), W), lambda: p.project(x[0], W),
                 lambda: p.project(x, W, ad[:3], A, B), lambda: p.project(x, W, ad, A[:1], B), lambda: p.project(x, W, ad),
                 lambda: p.project(x, W, A=A, B=B), lambda: p.project(x[:1].expand(4, 64), W),
                 lambda: p.project(x, W, out=torch.empty((4, 31), dtype=b)),
                 lambda: p.expert_project(x, W[None], off), lambda: p.expert_project(x, W, off),
                 lambda: p.expert_project(x, W[None, :31], off[:2], gate=True),
                 lambda: p.expert_project(x, W[None], off[:2], rows=ad.view(2, 2)),
                 lambda: p.expert_project(x[:0], W[None], off[:2], rows=ad),
                 lambda: p.route(torch.zeros((4, 8)), 9), lambda: p.route(torch.zeros((4, 8)), 0),
                 lambda: p.route(torch.zeros((4, 600)), 2), lambda: p.route(torch.zeros((4, 8, 1)), 2),
                 lambda: p.expert_combine(x, ad.view(2, 2), torch.zeros((2, 3))), lambda: p.expert_combine(x, ad, torch.zeros(4))):
        with pytest.raises(ValueError):
            call()


def test_binding_refuses_cpu_tensors(p):
    b = torch.bfloat16
    x, W = torch.zeros((4, 64), dtype=b), torch.zeros((32, 64), dtype=b)
    off = torch.zeros(2, dtype=torch.int32)
    for call in (lambda: p.project(x, W), lambda: p.expert_project(x, W[None], off), lambda: p.route(torch.zeros((4, 8)), 2),
                 lambda: p.expert_combine(x, off.view(1, 2), torch.zeros((1, 2)))):
        with pytest.raises(ValueError, match="GPU"):
            call()


def test_calls_with_too_many_threads_are_refused_before_any_launch(p):
    """A product whose last kernel needs 2^32 threads or more: refused whole, its first kernels (A x, the first of its
    tokens) are not launched either."""
    lib = p.library()
    for change in (dict(T=4, K=8, N=1 << 28),  # tiles of 8 tokens, after A x
                   dict(T=1, K=8, N=1 << 29), dict(T=1, K=8, N=1 << 29, adapter=None),
                   dict(T=264, K=72, N=(1 << 28) + 256)):  # 256 tokens in wide tiles, 8 by themselves
        call = project_args(**change, ldx=change["K"], ldo=change["N"], work_bytes=1 << 60)
        assert lib.hc_project(*call) == SIZE, change


def test_binding_takes_a_single_column_of_any_stride(p):
    """A column's own stride means nothing, as a single row's: the calls get as far as the tensors' device."""
    one = torch.zeros(24, dtype=torch.bfloat16).as_strided((4, 1), (6, 3))
    pos, w = torch.zeros((4, 1), dtype=torch.int32), torch.zeros((4, 1))
    x, W = torch.zeros((4, 64), dtype=torch.bfloat16), torch.zeros((1, 64), dtype=torch.bfloat16)
    for call in (lambda: p.expert_combine(one, pos, w), lambda: p.expert_combine(one, pos, w, out=one), lambda: p.route(one, 1),
                 lambda: p.project(x, W, out=one)):
        with pytest.raises(ValueError, match="GPU"):
            call()


def test_work_sizes_stay_under_their_bounds(p):
    """The most that the header promises for any sizes: a caller may make one scratch of it."""
    lib, rng = p.library(), random.Random(7)
    spread = lambda low, high: round(math.exp(rng.uniform(math.log(low), math.log(high))))  # noqa: E731
    most = 0
    for _ in range(20000):
        T, K, N, rank = spread(1, 100000), 8 * spread(1, 4096), spread(1, 60000), 8 * rng.randint(0, 16)
        size = lib.hc_project_work(T, K, N, rank)
        assert 0 <= size <= 32 * T * N + (16 * T * (rank + 8) if rank else 0), (T, K, N, rank)
        most = max(most, size / (32 * T * N))
        T, E, k = spread(1, 10 ** 7), spread(1, 512), rng.randint(1, 32)
        if T * k < 2 ** 31 - 65536:
            assert 0 <= lib.hc_route_work(T, E, k) <= 2048 * E, (T, E, k)
    assert most > 0.9  # (8 splits occur)
