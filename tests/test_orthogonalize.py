"""Orthogonalised update against the definition in 64 bits.

Tolerances, on the Frobenius norm of the error over that of the result.
float32 (and float16 before its last rounding): factors carry 22 bits, sums 32;
a step multiplies what the last one left by at most a = 3.4445 where singular
values are small and by p'(1.2) = 3.9 where they are near one, so roundings of
relative size 2^-22 at the start reach 484 2^-22 over sqrt(p) of the result (X_0
has norm one, the result about sqrt(p)), and those of the later steps, of
relative size 2^-21 with growth 3.9, 1.6 and so on, some 32 2^-21.  bfloat16:
factors of 11 bits; three roundings a step of rms 2^-12 times |b A + c A^2| <=
2.75, growing by 1.6 a step at rms: 16.0 2.75 2^-12 = 1.1e-2, and the output's
own 2^-9."""
import ctypes

import numpy as np
import pytest

from symmetric_tridiagonal_eigensolver_gb300 import bstq

COEFS = [(3.4445, -4.7750, 2.0315)] * 5


def reference(G, coefs=COEFS):
    X = G.astype(np.float64)
    tall = X.shape[-2] > X.shape[-1]
    if tall:
        X = np.swapaxes(X, -1, -2)
    norm = np.sqrt((X * X).sum((-1, -2), keepdims=True))
    X = np.divide(X, norm, out=np.zeros_like(X), where=norm > 0)
    for a, b, c in coefs:
        A = X @ np.swapaxes(X, -1, -2)
        X = a * X + (b * A + c * (A @ A)) @ X
    return np.swapaxes(X, -1, -2) if tall else X


def bound(dtype, p):
    exact = 484 * 2.0 ** -22 / p ** 0.5 + 32 * 2.0 ** -21
    return {"float32": exact, "float16": exact + 2.0 ** -11, "bfloat16": 1.1e-2 + 2.0 ** -9}[dtype]


def check(X, G, dtype, coefs=COEFS, scale=1.0):
    got, want = X.double().cpu().numpy(), reference(G.double().cpu().numpy() * scale, coefs)
    assert np.isfinite(got).all()
    err = np.sqrt(((got - want) ** 2).sum((-1, -2)))
    size = np.sqrt((want ** 2).sum((-1, -2)))
    lim = bound(dtype, min(G.shape[-2:])) * size
    assert (err <= lim).all(), (err / np.maximum(size, 1e-300)).max()


def matrices(batch, m, n, dtype, seed=0, kind="gradient"):
    import torch
    g = torch.Generator().manual_seed(seed)
    v = torch.randn(batch, m, n, generator=g)
    k = max(1, min(m, n) // 8)
    if kind == "gradient":
        v = torch.randn(batch, m, k, generator=g) @ torch.randn(batch, k, n, generator=g) / k ** 0.5 + 0.5 * v
    return v.to(getattr(torch, dtype)).cuda()


SIZES = [(3, 1, 1), (2, 1, 40), (2, 40, 1), (5, 3, 5), (4, 17, 16), (3, 31, 33), (7, 64, 64), (2, 65, 63), (3, 127, 129),
         (2, 128, 128), (2, 128, 300), (1, 129, 128), (2, 200, 77), (1, 256, 256), (1, 257, 513), (2, 513, 130),
         (1, 96, 1500), (1, 777, 640), (1, 1024, 1024), (1, 1100, 1031)]


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", ["float32", "bfloat16", "float16"])
@pytest.mark.parametrize("batch,m,n", SIZES)
@pytest.mark.parametrize("kind", ["gradient", "normal"])
def test_result(batch, m, n, dtype, kind):
    G = matrices(batch, m, n, dtype, seed=m + n, kind=kind)
    check(bstq.orthogonalize(G), G, dtype)


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", ["float32", "bfloat16"])
@pytest.mark.parametrize("batch,n", [(300, 32), (1030, 64), (40, 128)])
def test_large_batches(batch, n, dtype):
    G = matrices(batch, n, n, dtype, seed=n)
    check(bstq.orthogonalize(G), G, dtype)


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", ["float32", "bfloat16"])
@pytest.mark.parametrize("batch,m,n", [(1, 2048, 2048), (1, 2311, 2900), (3, 1500, 1200), (1, 4100, 1990)])
def test_large(batch, m, n, dtype):
    """Sizes whose tiles are worked on by pairs of blocks; the reference runs in
    64 bits on the GPU (torch's products)."""
    import torch
    G = matrices(batch, m, n, dtype, seed=m + n)
    X = G.double()
    X = X.transpose(1, 2) if m > n else X
    X = X / X.square().sum((1, 2), keepdim=True).sqrt()
    for a, b, c in COEFS:
        A = X @ X.transpose(1, 2)
        X = a * X + (b * A + c * (A @ A)) @ X
    X = X.transpose(1, 2) if m > n else X
    err = (bstq.orthogonalize(G).double() - X).square().sum((1, 2)).sqrt() / X.square().sum((1, 2)).sqrt()
    assert (err <= bound(dtype, min(m, n))).all(), err


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", ["float32", "bfloat16", "float16"])
@pytest.mark.parametrize("batch,m,n", [(1, 64, 4000), (2, 4096, 128), (1, 100, 2100), (9, 17, 3001), (1, 128, 4097)])
def test_few_rows_and_many_columns(batch, m, n, dtype):
    """One matrix to a cluster of 16 blocks, stacked ones too, and just beyond."""
    G = matrices(batch, m, n, dtype, seed=m + n)
    check(bstq.orthogonalize(G), G, dtype)


@pytest.mark.gpu
@pytest.mark.parametrize("steps", [1, 2, 8])
@pytest.mark.parametrize("m,n", [(60, 90), (300, 200)])
def test_steps_and_coefficients(steps, m, n):
    """Any number of steps, one set of coefficients for all or one for each;
    with (15/8, -10/8, 3/8) the iteration has the polar factor as its limit."""
    G = matrices(2, m, n, "float32", seed=3, kind="normal")
    check(bstq.orthogonalize(G, steps=steps), G, "float32", COEFS[:1] * steps)
    own = [(15 / 8, -10 / 8, 3 / 8)] * steps
    check(bstq.orthogonalize(G, steps=steps, coefs=own[0]), G, "float32", own)
    own = [(3.0 - 0.1 * k, -3.0 + 0.2 * k, 1.0 - 0.1 * k) for k in range(steps)]
    check(bstq.orthogonalize(G, steps=steps, coefs=own), G, "float32", own)


@pytest.mark.gpu
@pytest.mark.parametrize("m,n", [(48, 48), (100, 400)])
def test_the_limit_is_the_polar_factor(m, n):
    """Twenty-four convergent steps against U V^T of numpy's SVD."""
    G = matrices(1, m, n, "float32", seed=3, kind="gradient")
    X = bstq.orthogonalize(G[0], steps=24, coefs=(15 / 8, -10 / 8, 3 / 8)).double().cpu().numpy()
    u, s, vt = np.linalg.svd(G[0].double().cpu().numpy(), full_matrices=False)
    assert s[-1] / np.sqrt((s * s).sum()) > 1e-5  # well inside what 24 steps reach: 1.875^17 > 4e4
    # roundings of the start grow by s_max / s_min on their way
    assert np.abs(X - u @ vt).max() <= 2.0 ** -19 * s[0] / s[-1] + 1e-5


@pytest.mark.gpu
@pytest.mark.parametrize("m,n", [(40, 56), (200, 150)])
@pytest.mark.parametrize("dtype", ["float32", "bfloat16"])
def test_scale_does_not_matter(m, n, dtype):
    """Up to where |G|^2 leaves 32 bits, both ways; powers of two give equal bits."""
    import torch
    G = matrices(2, m, n, dtype, seed=5)
    X = bstq.orthogonalize(G)
    for k in (-100, -60, -40, 40, 60, 100):
        assert torch.equal(bstq.orthogonalize(G * 2.0 ** k), X), k


@pytest.mark.gpu
def test_half_precision_extremes():
    G = matrices(1, 70, 90, "float16", seed=5)
    check(bstq.orthogonalize(G * 2.0 ** -12), G * 2.0 ** -12, "float16")
    check(bstq.orthogonalize(G * 2.0 ** 12), G * 2.0 ** 12, "float16")


@pytest.mark.gpu
@pytest.mark.parametrize("n", [24, 160])
def test_zero_and_non_finite_matrices_stand_alone(n):
    import torch
    G = matrices(5, n, n + 8, "float32", seed=6)
    want = bstq.orthogonalize(G)
    G[1] = 0
    G[2, 3, 4] = float("nan")
    G[3, n - 1, 0] = float("inf")
    X = bstq.orthogonalize(G)
    assert (X[1] == 0).all() and torch.isnan(X[2]).all() and torch.isnan(X[3]).all()
    assert torch.equal(X[0], want[0]) and torch.equal(X[4], want[4])


SUMS = pytest.mark.xfail(reason="the bound counts the factors' roundings; at 300 terms those of the 32-bit sums are "
                                "larger in the directions of zero singular values, see the next test", strict=False)


@pytest.mark.gpu
@pytest.mark.parametrize("m,n", [(50, 70), (130, 70), pytest.param(300, 300, marks=SUMS)])
@pytest.mark.parametrize("rank", [1, 3])
def test_rank_deficient(m, n, rank):
    """Zero singular values stay zero: the iteration only scales what is there."""
    import torch
    g = torch.Generator().manual_seed(1)
    G = (torch.randint(-3, 4, (m, rank), generator=g) @ torch.randint(-3, 4, (rank, n), generator=g)).float().cuda()
    check(bstq.orthogonalize(G[None]), G[None], "float32")


@pytest.mark.gpu
@pytest.mark.parametrize("m,n,rank", [(300, 300, 1), (300, 300, 3), (600, 200, 2), (150, 900, 5)])
def test_rank_deficient_with_the_sums_roundings(m, n, rank):
    """A sum of K terms in 32 bits is off by some sqrt(K) 2^-23 of its size.  In
    B X (of |b A + c A^2| = 2.75 times X) that lands in the directions of zero
    singular values too, and each later step multiplies it by 3.4445: 140 times
    from the first step on, 197 over all; the result has norm sqrt(rank)."""
    import torch
    g = torch.Generator().manual_seed(2)
    G = (torch.randint(-3, 4, (m, rank), generator=g) @ torch.randint(-3, 4, (rank, n), generator=g)).float().cuda()
    X = bstq.orthogonalize(G).double().cpu().numpy()
    want = reference(G.double().cpu().numpy())
    terms = min(m, n)
    lim = (484 * 2.0 ** -22 + 2.75 * 197 * 2.0 ** -23 * terms ** 0.5) / rank ** 0.5 + 32 * 2.0 ** -21
    assert np.linalg.norm(X - want) <= lim * np.linalg.norm(want)


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", ["float32", "bfloat16"])
@pytest.mark.parametrize("m,n", [(30, 50), (130, 70), (260, 512)])
def test_layouts(m, n, dtype):
    import torch
    G = matrices(3, m, n, dtype, seed=8)
    want = bstq.orthogonalize(G)
    wide = torch.full((3, m + 2, n + 5), float("nan"), dtype=G.dtype, device="cuda")
    view = wide[:, 1:1 + m, 3:3 + n]
    view.copy_(G)
    out = torch.full((3, m + 2, n + 5), 7.0, dtype=G.dtype, device="cuda")
    got = bstq.orthogonalize(view, out=out[:, 1:1 + m, 3:3 + n])
    assert torch.equal(got, want)
    rim = out.clone()
    rim[:, 1:1 + m, 3:3 + n] = 7.0
    assert (rim == 7.0).all()
    flipped = G.transpose(1, 2).contiguous().transpose(1, 2)
    check(bstq.orthogonalize(flipped), G, dtype)
    assert torch.equal(bstq.orthogonalize(G[1]), want[1])                       # one matrix, no batch axis
    assert torch.equal(bstq.orthogonalize(G[:1].expand(3, m, n))[2], want[0])   # batch stride zero
    bstq.orthogonalize(G, out=G)                                                # in place
    assert torch.equal(G, want)


@pytest.mark.gpu
def test_equal_inputs_give_equal_bits():
    import torch
    for size in ((40, 64, 64), (2, 300, 500)):
        G = matrices(*size, "bfloat16", seed=4)
        X = bstq.orthogonalize(G)
        for _ in range(4):
            assert torch.equal(bstq.orthogonalize(G), X)


@pytest.mark.gpu
@pytest.mark.parametrize("batch,m,n", [(30, 64, 64), (1, 300, 400)])
def test_stream_workspace_and_graph(batch, m, n):
    import torch
    G = matrices(batch, m, n, "float32", seed=4)
    want = bstq.orthogonalize(G)
    work = torch.full((bstq.load().bstq_orthogonalize_work_size(bstq.F32, batch, m, n),), 255, dtype=torch.uint8,
                      device="cuda")
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    for _ in range(2):
        X = bstq.orthogonalize(G, work=work, stream=side)
        side.synchronize()
        assert torch.equal(X, want)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        X = bstq.orthogonalize(G, work=work)
    G.copy_(matrices(batch, m, n, "float32", seed=9))
    graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(X, bstq.orthogonalize(G))


@pytest.mark.gpu
def test_empty_and_refusals_of_the_binding():
    import torch
    assert bstq.orthogonalize(torch.empty(0, 4, 5, device="cuda")).shape == (0, 4, 5)
    assert bstq.orthogonalize(torch.empty(3, 0, 5, device="cuda")).shape == (3, 0, 5)
    G = torch.zeros(2, 4, 6, device="cuda")
    for kind, args, kw in (
            (TypeError, (G.double(),), {}), (ValueError, (G.cpu(),), {}), (ValueError, (G[0, 0],), {}),
            (ValueError, (G,), {"steps": 0}), (ValueError, (G,), {"steps": 33}), (ValueError, (G,), {"coefs": (1, 2)}),
            (ValueError, (G,), {"coefs": [(1.0, 2.0, 3.0)] * 4}), (ValueError, (G,), {"coefs": (float("nan"), 0, 0)}),
            (ValueError, (G,), {"coefs": (17.0, 0, 0)}), (ValueError, (G,), {"out": G[:1]}),
            (ValueError, (G,), {"out": G.half()}), (ValueError, (G[:, ::2, ::2],), {}),
            (ValueError, (G,), {"out": G[:1].expand(2, 4, 6)}),
            (ValueError, (G,), {"work": torch.empty(8, dtype=torch.uint8, device="cuda")})):
        with pytest.raises(kind):
            bstq.orthogonalize(*args, **kw)


def test_refusals_of_the_library():
    import os
    if not os.path.exists(bstq.LIB_PATH):
        from symmetric_tridiagonal_eigensolver_gb300 import build
        build.build()
    lib = bstq.load()
    buf = (ctypes.c_char * 4096)()
    base = ctypes.addressof(buf) + (-ctypes.addressof(buf)) % 256
    p, odd = ctypes.c_void_p(base), ctypes.c_void_p(base + 1)
    nan, large = (ctypes.c_float * 15)(*([float("nan")] * 15)), (ctypes.c_float * 15)(*([17.0] * 15))
    neg, lap = (ctypes.c_int64 * 4)(24, -6, 24, 6), (ctypes.c_int64 * 4)(24, 6, 24, 5)
    good = [0, 2, 4, 6, p, p, None, 5, None, p, None]
    for k, value, code in [(0, 1, -1), (0, 9, -1), (1, -1, -2), (1, 65536, -2), (2, -1, -3), (2, 1 << 21, -3),
                           (3, -1, -4), (3, 1 << 21, -4), (4, None, -5), (4, odd, -5), (5, None, -6), (6, neg, -7),
                           (6, lap, -7), (7, 0, -8), (7, 33, -8), (8, nan, -9), (8, large, -9), (9, None, -10),
                           (9, odd, -10), (1, 0, 0), (2, 0, 0), (3, 0, 0)]:
        args = list(good)
        args[k] = value
        assert lib.bstq_orthogonalize(*args) == code, (k, value)
    size = lib.bstq_orthogonalize_work_size
    assert size(1, 2, 4, 6) == 0 and size(0, -1, 4, 6) == 0 and size(0, 1, 1 << 21, 6) == 0
    assert size(0, 0, 4, 6) >= 256 and size(2, 3, 4, 6) >= 256
    import torch
    if not torch.cuda.is_available():
        assert lib.bstq_orthogonalize(*good) == bstq.ERR_NODEVICE


@pytest.mark.gpu
@pytest.mark.parametrize("m,n,kind", [(1531, 777, "gradient"), (2048, 2048, "gradient"), (128, 128, "gradient"),
                                      (128, 4096, "gradient"), (90, 600, "graded"), (700, 900, "graded")])
def test_scale_does_not_matter_at_any_exponent(m, n, kind):
    """Every power of two at which G's values stay normal: the sums of squares
    that blocks, warps and clusters join must neither overflow nor change a
    rounding.  "graded": rows of very different sizes, whose sums are taken in
    different ranges."""
    import torch
    G = matrices(1, m, n, "float32", seed=5, kind="gradient")
    if kind == "graded":
        G = G * (2.0 ** -(5.0 * (torch.arange(m, device="cuda") % 8)))[:, None]
    want = bstq.orthogonalize(G)
    assert torch.isfinite(want).all()
    if kind == "gradient":
        check(want, G, "float32")
    bad = [k for k in range(-60 if kind == "graded" else -100, 121)
           if not torch.equal(bstq.orthogonalize(G * 2.0 ** k), want)]
    assert not bad, bad


@pytest.mark.gpu
def test_norm_of_the_largest_and_smallest_values():
    """All values at float32's ends, where no square and hardly a value fits."""
    import torch
    for size in ((1, 100, 130), (1, 300, 260)):
        sign = torch.where(torch.randn(size, generator=torch.Generator().manual_seed(1)) > 0, 1.0, -1.0).cuda()
        want = bstq.orthogonalize(sign)
        for top in (3.0e38, 2.0 ** -149, 2.0 ** -140):
            assert torch.allclose(bstq.orthogonalize(sign * top), want, rtol=0, atol=2e-6), top


def test_results_whose_rows_overlap_are_refused():
    import os
    if not os.path.exists(bstq.LIB_PATH):
        from symmetric_tridiagonal_eigensolver_gb300 import build
        build.build()
    lib = bstq.load()
    buf = (ctypes.c_char * 4096)()
    p = ctypes.c_void_p(ctypes.addressof(buf) + (-ctypes.addressof(buf)) % 256)
    for xb, xr in ((6, 6), (12, 6), (23, 6), (8, 13), (6, 17)):
        assert lib.bstq_orthogonalize(0, 3, 4, 6, p, p, (ctypes.c_int64 * 4)(24, 6, xb, xr), 5, None, p, None) == -7, (xb, xr)
    import torch
    if not torch.cuda.is_available():
        for xb, xr in ((24, 6), (25, 6), (6, 18), (30, 7), (40, 6)):
            assert lib.bstq_orthogonalize(0, 3, 4, 6, p, p, (ctypes.c_int64 * 4)(24, 6, xb, xr), 5, None, p,
                                          None) == bstq.ERR_NODEVICE, (xb, xr)


def test_sizes_go_in_tiles_where_no_cluster_fits_them(tmp_path):
    """A device, or a part of one, may place fewer blocks to a cluster than 16:
    the sizes that need more are not small there (the workspace and the launch
    ask the same function)."""
    import os
    import shutil
    import subprocess
    gxx = shutil.which("g++")
    if gxx is None:
        pytest.skip("g++ not available")
    root = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
    exe = str(tmp_path / "orth_plan_check")
    subprocess.run([gxx, "-std=c++17", "-O1", "-Wall", "-Werror", "-I",
                    os.path.join(root, "symmetric_tridiagonal_eigensolver_gb300", "csrc"),
                    os.path.join(root, "tests", "orth_plan_check.cpp"), "-o", exe], check=True)
    cases = [((128, 4096, 16), (1, 16)), ((4096, 128, 16), (1, 16)), ((128, 4097, 16), (0, 32)), ((129, 200, 16), (0, 1)),
             ((128, 4097, 32), (0, 32)), ((128, 4096, 8), (0, 16)), ((64, 2048, 8), (1, 8)), ((2049, 64, 8), (0, 16)),
             ((1, 1024, 4), (1, 4)), ((100, 1025, 4), (0, 8)), ((128, 256, 1), (1, 1)), ((128, 257, 1), (0, 2)),
             ((1, 1, 1), (1, 1)), ((1 << 20, 1, 16), (0, 4096))]
    r = subprocess.run([exe], input="".join("%d %d %d\n" % c for c, _ in cases), capture_output=True, text=True, timeout=60,
                       check=True)
    assert [tuple(map(int, line.split())) for line in r.stdout.splitlines()] == [want for _, want in cases]


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", ["float32", "bfloat16"])
@pytest.mark.parametrize("batch,m,n", [(30, 64, 64), (3, 100, 900), (2, 128, 4000), (1, 150, 200), (2, 300, 260)])
def test_a_wait_that_runs_out_leaves_no_wrong_numbers(batch, m, n, dtype):
    """With no cycles to wait, whether a wait runs out is up to the products' time:
    the status says it, and each result is right or NaN."""
    import torch
    lib = bstq.load()
    G = matrices(batch, m, n, dtype, seed=2)
    want = bstq.orthogonalize(G)
    code = {"float32": bstq.F32, "bfloat16": bstq.BF16}[dtype]
    work = torch.zeros(lib.bstq_orthogonalize_work_size(code, batch, m, n), dtype=torch.uint8, device="cuda")
    status = work[:4].view(torch.int32)
    torch.cuda.synchronize()
    before = lib.bstq_set_wait_limit(0)
    try:
        for _ in range(3):
            X = bstq.orthogonalize(G, work=work)
            torch.cuda.synchronize()
            gone = torch.isnan(X)
            assert bool((gone | (X == want)).all())
            assert int(status) == 1 or not bool(gone.any())
    finally:
        lib.bstq_set_wait_limit(before)
    assert torch.equal(bstq.orthogonalize(G, work=work), want) and int(status) == 0


STEEP = [(8.3, -23.6, 17.3), (4.1, -2.9, 0.55), (3.9, -2.8, 0.5), (3.3, -2.4, 0.46), (2.3, -1.6, 0.4)]


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", ["float32", "bfloat16"])
@pytest.mark.parametrize("m,n", [(64, 64), (100, 700), (300, 260)])
def test_a_schedule_with_a_steep_first_step(m, n, dtype):
    """Coefficients above 16 in b and c.  Roundings of the start grow by the product
    of the a (1007 instead of 484), those of the products by |b A + c A^2| <= 8.05
    instead of 2.75."""
    G = matrices(2, m, n, dtype, seed=11, kind="normal")
    X = bstq.orthogonalize(G, coefs=STEEP).double().cpu().numpy()
    want = reference(G.double().cpu().numpy(), STEEP)
    later = 8.05 / 2.75 * (32 * 2.0 ** -21 if dtype == "float32" else 1.1e-2)
    lim = 1007 * 2.0 ** -22 / min(m, n) ** 0.5 + later + (0 if dtype == "float32" else 2.0 ** -9)
    assert np.linalg.norm(X - want) <= lim * np.linalg.norm(want)


def test_limits_of_the_coefficients():
    import os
    if not os.path.exists(bstq.LIB_PATH):
        from symmetric_tridiagonal_eigensolver_gb300 import build
        build.build()
    lib = bstq.load()
    buf = (ctypes.c_char * 4096)()
    p = ctypes.c_void_p(ctypes.addressof(buf) + (-ctypes.addressof(buf)) % 256)
    import torch
    for row, code in (((16.5, 0, 0), -9), ((0, 32.5, 0), -9), ((0, 0, -32.5), -9), ((0, 0, float("inf")), -9),
                      ((8.3, -23.6, 17.3), bstq.ERR_NODEVICE), ((16, 32, -32), bstq.ERR_NODEVICE)):
        if code != -9 and torch.cuda.is_available():
            continue  # these pointers are no device memory
        c = (ctypes.c_float * 3)(*row)
        assert lib.bstq_orthogonalize(0, 2, 4, 6, p, p, None, 1, c, p, None) == code, row


def plain32(G):
    """The same products in torch's 32 bits, rounded once at the end."""
    X = G.float()
    tall = X.shape[-2] > X.shape[-1]
    X = X.mT if tall else X
    X = X / X.square().sum((-1, -2), keepdim=True).sqrt()
    for a, b, c in COEFS:
        A = X @ X.mT
        X = a * X + (b * A + c * (A @ A)) @ X
    return (X.mT if tall else X).to(G.dtype)


def low_rank(m, n, rank, dtype, seed):
    import torch
    g = torch.Generator().manual_seed(seed)
    G = torch.randint(-3, 4, (m, rank), generator=g) @ torch.randint(-3, 4, (rank, n), generator=g)
    return G.to(getattr(torch, dtype)).cuda()


@pytest.mark.gpu
@pytest.mark.parametrize("m,n", [(64, 64), (128, 128), (300, 300), (600, 200), (150, 900), (128, 1024), (777, 1531)])
@pytest.mark.parametrize("rank", [1, 3])
def test_rank_deficient_is_as_exact_as_plain_products(m, n, rank):
    """Zero singular values amplify every rounding of the products by 3.4445 a
    step, whoever computes them: the mean error over eight matrices stays below
    twice that of the same products in plain 32 bits.  (Dropped second terms of
    the factors would leave 2^-12 times 197, a hundred times more.)"""
    mine = plain = 0.0
    for seed in range(8):
        G = low_rank(m, n, rank, "float32", seed)
        want = reference(G.double().cpu().numpy())
        size = np.linalg.norm(want)
        mine += np.linalg.norm(bstq.orthogonalize(G).double().cpu().numpy() - want) / size
        plain += np.linalg.norm(plain32(G).double().cpu().numpy() - want) / size
    assert mine <= 2 * plain, (mine / 8, plain / 8)


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", ["bfloat16", "float16"])
@pytest.mark.parametrize("m,n", [(20, 30), (64, 64), (128, 1024), (300, 300), (600, 200)])
@pytest.mark.parametrize("rank", [1, 3])
def test_rank_deficient_in_16_bits(m, n, rank, dtype):
    """The bounds of full rank and, for half, the 32-bit sums' (as above)."""
    sums = 2.75 * 197 * 2.0 ** -23 * min(m, n) ** 0.5 / rank ** 0.5 if dtype == "float16" else 0.0
    for seed in range(3):
        G = low_rank(m, n, rank, dtype, seed)
        want = reference(G.double().cpu().numpy())
        err = np.linalg.norm(bstq.orthogonalize(G).double().cpu().numpy() - want) / np.linalg.norm(want)
        assert err <= bound(dtype, rank) + sums


@pytest.mark.gpu
@pytest.mark.parametrize("m,n", [(64, 64), (100, 90), (128, 1024), (512, 512), (1531, 777), (1100, 2900)])
@pytest.mark.parametrize("kind", ["gradient", "normal"])
def test_bf16_error_is_near_the_outputs_rounding(m, n, kind):
    """Factors of 11 bits, eight times finer than the result: three roundings of
    2^-12 a step, grown to some 0.9e-3 at 1024 rows and more in fewer, next to the
    result's own 1.66e-3: together below twice the latter."""
    import torch
    G = matrices(1, m, n, "bfloat16", seed=m + n, kind=kind)[0]
    want = torch.from_numpy(reference(G.double().cpu().numpy())).cuda()
    rounding = float((want.to(torch.bfloat16).double() - want).norm())
    assert float((bstq.orthogonalize(G).double() - want).norm()) <= 2 * rounding
