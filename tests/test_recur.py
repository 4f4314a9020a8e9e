"""Gated linear recurrence, its gradients and its single-token form, against
the definitions in 64 bits.

Tolerances.  A state is a convex combination of h0 and the inputs, so with
M = max(|x|, |h0|) every state is at most M.  One step in 32 bits (u = 2^-24)
adds a rounding of at most u M, and the gate's relative error (below 8 u: the
exponentials, the reciprocal and the products) enters times (1 - a) 2 M; the
second sums to 16 u M over a whole sequence, since the (1 - a_t) times the later decays
telescope to one, and the first, with independent signs, to 8 sqrt(T) u M with
a wide margin.  States: (32 + 8 sqrt(T)) u M, plus half a unit in the last
place of the output's type.  The same holds for g with its own largest value,
and products of it add a few u of their factors' largest values."""
import ctypes

import numpy as np
import pytest

from symmetric_tridiagonal_eigensolver_gb300 import bstq

U = 2.0 ** -24
HALF = {"float32": 2.0 ** -24, "bfloat16": 2.0 ** -8, "float16": 2.0 ** -10}  # a whole unit, for safety at ties
TINY = {"float32": 0.0, "bfloat16": 0.0, "float16": 2.0 ** -24}               # float16's subnormal spacing


def reference(x, r, rate, h0=None, lengths=None):
    """(h, hT) in float64, step by step."""
    B, T, D = x.shape
    s = 1 / (1 + np.exp(-r))
    z = np.maximum(rate, 0) * s
    a, q = np.exp(-z), -np.expm1(-z)
    h = np.zeros((B, T, D))
    last = np.zeros((B, D)) if h0 is None else h0.astype(np.float64).copy()
    for b in range(B):
        for t in range(T if lengths is None else min(max(int(lengths[b]), 0), T)):
            last[b] = a[b, t] * last[b] + q[b, t] * x[b, t]
            h[b, t] = last[b]
    return h, last


def reference_grad(x, r, rate, h, dh, dhT=None, h0=None, lengths=None):
    """(dx, dr, drate, dh0, largest |g|, sum of |dz s|) in float64."""
    B, T, D = x.shape
    s = 1 / (1 + np.exp(-r))
    lam = np.maximum(rate, 0)
    a, q = np.exp(-lam * s), -np.expm1(-lam * s)
    dx, dr, drate, mass = np.zeros_like(x), np.zeros_like(x), np.zeros(D), np.zeros(D)
    g = np.zeros((B, D)) if dhT is None else dhT.astype(np.float64).copy()
    top = np.abs(g).max(initial=0.0)
    for b in range(B):
        for t in range((T if lengths is None else min(max(int(lengths[b]), 0), T)) - 1, -1, -1):
            before = h[b, t - 1] if t else (h0[b] if h0 is not None else 0.0)
            g[b] += dh[b, t]
            top = max(top, np.abs(g[b]).max(initial=0.0))
            dz = a[b, t] * g[b] * (x[b, t] - before)
            dx[b, t] = q[b, t] * g[b]
            dr[b, t] = dz * lam * s[b, t] * (1 - s[b, t])
            drate += dz * s[b, t]
            mass += np.abs(dz * s[b, t])
            g[b] = a[b, t] * g[b]
    return dx, dr, np.where(rate > 0, drate, 0.0), g, top, mass


def chain_rates(D, scale=1.0):
    """Eigenvalues of tridiag(-1; 2): rates from nearly none to four times the scale."""
    return (scale * (2 - 2 * np.cos(np.arange(1, D + 1) * np.pi / (D + 1)))).astype(np.float32)


def problem(B, T, D, dtype, seed=0, layout="dense"):
    import torch
    g = torch.Generator().manual_seed(seed)

    def make(*shape, shift=0.0, scale=1.0):
        v = (scale * torch.randn(*shape, generator=g) + shift).to(getattr(torch, dtype))
        if layout == "dense":
            return v.cuda()
        if layout == "time_major":  # (T, B, D) storage
            return v.cuda().transpose(0, 1).contiguous().transpose(0, 1)
        if layout == "wide":        # rows inside wider rows, starting off any 16-byte boundary
            w = torch.full((shape[0], shape[1], shape[2] + 5), float("nan"), dtype=v.dtype, device="cuda")
            w[:, :, 3:3 + shape[2]] = v.cuda()
            return w[:, :, 3:3 + shape[2]]
        raise AssertionError(layout)

    return make, g


def f64(t):
    return t.detach().double().cpu().numpy()


def near(got, want, bound, dtype):
    err = np.abs(f64(got) - want)
    lim = bound + HALF[dtype] * np.abs(want) + TINY[dtype]
    assert np.isfinite(f64(got)).all()
    assert (err <= lim).all(), (err - lim).max()


SHAPES = [(1, 1, 1), (2, 1, 33), (3, 2, 7), (2, 17, 96), (1, 63, 130), (2, 129, 65), (1, 257, 64), (3, 300, 31),
          (5, 64, 256), (1, 1025, 48), (2, 700, 1003), (1, 5000, 24), (1, 20000, 8)]


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", ["float32", "bfloat16", "float16"])
@pytest.mark.parametrize("B,T,D", SHAPES)
def test_states(B, T, D, dtype):
    import torch
    make, g = problem(B, T, D, dtype, seed=B * T + D)
    x, r = make(B, T, D), make(B, T, D, shift=-1.0, scale=1.5)
    rate = torch.from_numpy(chain_rates(D)).cuda()
    h0 = torch.randn(B, D, generator=g).cuda()
    h, hT = bstq.recur(x, r, rate, h0=h0)
    want, last = reference(f64(x), f64(r), f64(rate), f64(h0))
    m = max(np.abs(f64(x)).max(), np.abs(f64(h0)).max())
    tol = (32 + 8 * T ** 0.5) * U * m
    near(h, want, tol, dtype)
    near(hT, last, tol, "float32")
    h, hT = bstq.recur(x, r, rate)
    want, last = reference(f64(x), f64(r), f64(rate))
    near(h, want, tol, dtype)
    near(hT, last, tol, "float32")


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", ["float32", "bfloat16", "float16"])
@pytest.mark.parametrize("B,T,D", SHAPES)
def test_gradients(B, T, D, dtype):
    import torch
    make, g = problem(B, T, D, dtype, seed=B * T + D + 1)
    x, r, dh = make(B, T, D), make(B, T, D, shift=-1.0, scale=1.5), make(B, T, D)
    rate = torch.from_numpy(chain_rates(D, 0.7)).cuda()
    h0, dhT = torch.randn(B, D, generator=g).cuda(), torch.randn(B, D, generator=g).cuda()
    for k in range(2):
        kw = dict(h0=h0, dhT=dhT) if k == 0 else {}
        h, _ = bstq.recur(x, r, rate, h0=kw.get("h0"))
        dx, dr, drate, dh0 = bstq.recur_grad(x, r, rate, h, dh, **kw)
        want = reference_grad(f64(x), f64(r), f64(rate), f64(h), f64(dh), f64(dhT) if k == 0 else None,
                              f64(h0) if k == 0 else None)
        check_gradients((dx, dr, drate, dh0), want, f64(x), f64(h), f64(h0), T, dtype)


def check_gradients(got, want, x, h, h0, T, dtype):
    dx, dr, drate, dh0 = got
    wx, wr, wrate, w0, top, mass = want
    rel = (32 + 8 * T ** 0.5) * U
    swing = np.abs(x).max(initial=0.0) + max(np.abs(h).max(initial=0.0), np.abs(h0).max(initial=0.0))
    near(dx, wx, rel * top, dtype)
    near(dh0, w0, rel * top, "float32")
    near(dr, wr, 2 * rel * top * swing, dtype)  # lambda s (1 - s) a is below one for rates up to four
    # each term's relative part, and a sum of N terms in any fixed order: log2 N + one run of steps
    terms = x.shape[0] * T
    err = np.abs(f64(drate) - wrate)
    lim = 2 * rel * top * swing * terms ** 0.5 + 64 * U * mass + 1e-30
    assert (err <= lim).all(), (err - lim).max()


@pytest.mark.gpu
def test_gradients_against_differences():
    """Directional differences of the 64-bit recurrence, step 1e-5: their own
    error is of order 1e-9, the kernel's that of its states and gradients."""
    import torch
    B, T, D = 2, 70, 40
    make, g = problem(B, T, D, "float32", seed=5)
    x, r, dh = make(B, T, D), make(B, T, D), make(B, T, D)
    rate = torch.from_numpy(chain_rates(D)).cuda()
    h0, dhT = torch.randn(B, D, generator=g).cuda(), torch.randn(B, D, generator=g).cuda()
    lengths = np.array([T, 41], dtype=np.int32)
    ln = torch.from_numpy(lengths).cuda()
    h, _ = bstq.recur(x, r, rate, h0=h0, lengths=ln)
    grads = bstq.recur_grad(x, r, rate, h, dh, dhT=dhT, h0=h0, lengths=ln)
    base = [f64(x), f64(r), f64(rate), f64(h0)]
    rng = np.random.default_rng(0)

    def loss(p):
        hh, last = reference(*p, lengths=lengths)
        return (hh * f64(dh)).sum() + (last * f64(dhT)).sum()

    for k in range(4):
        for _ in range(3):
            way = rng.standard_normal(base[k].shape)
            up, down = list(base), list(base)
            up[k], down[k] = base[k] + 1e-5 * way, base[k] - 1e-5 * way
            slope = (loss(up) - loss(down)) / 2e-5
            got = (f64(grads[k]) * way).sum()
            size = np.sqrt((f64(grads[k]) ** 2).sum() * (way ** 2).sum())
            assert abs(got - slope) <= 2e-5 * size + 1e-6


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", ["float32", "bfloat16"])
@pytest.mark.parametrize("T,D", [(1, 40), (50, 33), (700, 64), (1500, 258)])
def test_lengths_end_sequences_and_nothing_beyond_is_read(T, D, dtype):
    import torch
    lengths = [0, T, 1, T // 2, T - 1, -3, T + 9, min(T, 64), min(T, 65)]
    B = len(lengths)
    make, g = problem(B, T, D, dtype, seed=T)
    x, r, dh = make(B, T, D), make(B, T, D), make(B, T, D)
    n = np.clip(lengths, 0, T)
    for b in range(B):  # poison what lies beyond
        for v in (x, r, dh):
            v[b, n[b]:] = float("nan")
    rate = torch.from_numpy(chain_rates(D)).cuda()
    h0, dhT = torch.randn(B, D, generator=g).cuda(), torch.randn(B, D, generator=g).cuda()
    ln = torch.tensor(lengths, dtype=torch.int32, device="cuda")
    h, hT = bstq.recur(x, r, rate, h0=h0, lengths=ln)
    xs, rs, dhs = (np.nan_to_num(f64(v)) for v in (x, r, dh))
    want, last = reference(xs, rs, f64(rate), f64(h0), lengths)
    m = max(np.abs(xs).max(), np.abs(f64(h0)).max())
    tol = (32 + 8 * T ** 0.5) * U * m
    near(h, want, tol, dtype)
    near(hT, last, tol, "float32")
    for b in range(B):
        assert (h[b, n[b]:] == 0).all()
    assert torch.equal(hT[0], h0[0])
    hp = h.clone()
    for b in range(B):
        hp[b, n[b]:] = float("nan")
    dx, dr, drate, dh0 = bstq.recur_grad(x, r, rate, hp, dh, dhT=dhT, h0=h0, lengths=ln)
    ref = reference_grad(xs, rs, f64(rate), f64(h), dhs, f64(dhT), f64(h0), lengths)
    check_gradients((dx, dr, drate, dh0), ref, xs, f64(h), f64(h0), T, dtype)
    for b in range(B):
        assert (dx[b, n[b]:] == 0).all() and (dr[b, n[b]:] == 0).all()
    assert torch.equal(dh0[0], dhT[0])


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", ["float32", "bfloat16", "float16"])
@pytest.mark.parametrize("layout", ["time_major", "wide"])
@pytest.mark.parametrize("T,D", [(90, 64), (301, 57)])
def test_strides(T, D, layout, dtype):
    import torch
    B = 3
    make, g = problem(B, T, D, dtype, seed=9, layout=layout)
    x, r, dh, out = make(B, T, D), make(B, T, D), make(B, T, D), make(B, T, D)
    rate = torch.from_numpy(chain_rates(D)).cuda()
    dense = [v.contiguous() for v in (x, r, dh)]
    h, hT = bstq.recur(x, r, rate, out=out)
    hd, hTd = bstq.recur(dense[0], dense[1], rate)
    assert h is out
    want, last = reference(f64(x), f64(r), f64(rate))
    tol = (32 + 8 * T ** 0.5) * U * np.abs(f64(x)).max()
    near(h, want, tol, dtype)
    near(hT, last, tol, "float32")
    got = bstq.recur_grad(x, r, rate, h, dh)
    check_gradients(got, reference_grad(f64(x), f64(r), f64(rate), f64(h), f64(dh)), f64(x), f64(h),
                    np.zeros((B, D)), T, dtype)
    if layout == "wide":  # the elements between the rows stay as they were
        assert torch.isnan(out.as_strided((B, T, 2), out.stride(), out.storage_offset() + D)).all()


@pytest.mark.gpu
def test_broadcast_inputs_with_stride_zero():
    import torch
    B, T, D = 4, 70, 64
    make, _ = problem(1, T, D, "float32", seed=3)
    x, r = make(1, T, D), make(1, T, D)
    rate = torch.from_numpy(chain_rates(D)).cuda()
    h, _ = bstq.recur(x.expand(B, T, D), r.expand(B, T, D), rate)
    one, _ = bstq.recur(x, r, rate)
    assert all(torch.equal(h[b], one[0]) for b in range(B))


@pytest.mark.gpu
@pytest.mark.parametrize("T", [3, 400])
def test_rates_at_and_below_zero_hold_the_state(T):
    import torch
    B, D = 2, 64
    make, g = problem(B, T, D, "float32", seed=4)
    x, r, dh = make(B, T, D), make(B, T, D), make(B, T, D)
    rate = torch.tensor([0.0, -1e-7, -5.0, 1e-6] * (D // 4), device="cuda")
    h0 = torch.randn(B, D, generator=g).cuda()
    h, hT = bstq.recur(x, r, rate, h0=h0)
    held = rate <= 0
    assert torch.equal(h[:, :, held], h0[:, None, held].expand(B, T, int(held.sum())))
    assert torch.equal(hT[:, held], h0[:, held])
    dx, dr, drate, dh0 = bstq.recur_grad(x, r, rate, h, dh, h0=h0)
    assert (dx[:, :, held] == 0).all() and (dr[:, :, held] == 0).all() and (drate[held] == 0).all()
    assert (drate[~held] != 0).all()
    near(dh0[:, held], f64(dh)[:, :, held.cpu().numpy()].sum(1), (32 + 8 * T ** 0.5) * U * 4 * T ** 0.5, "float32")


@pytest.mark.gpu
def test_extreme_gates_and_rates():
    """Gates that are shut (the state holds) and open with a large rate (the
    state follows the input), at the ends of float32's range."""
    import torch
    B, T, D = 1, 200, 64
    make, g = problem(B, T, D, "float32", seed=8)
    x = make(B, T, D)
    r = torch.full((B, T, D), 40.0, device="cuda")
    r[:, :, ::2] = -200.0
    rate = torch.full((D,), 1e4, device="cuda")
    h0 = torch.randn(B, D, generator=g).cuda()
    h, hT = bstq.recur(x, r, rate, h0=h0)
    assert torch.equal(h[:, :, ::2], h0[:, None, ::2].expand(B, T, D // 2))
    assert torch.allclose(h[:, :, 1::2], x[:, :, 1::2], rtol=0, atol=2e-6)
    dx, dr, drate, dh0 = bstq.recur_grad(x, r, rate, h, x, h0=h0)
    for v in (dx, dr, drate, dh0):
        assert torch.isfinite(v).all()
    assert (dx[:, :, ::2] == 0).all() and (dr == 0).all()


@pytest.mark.gpu
@pytest.mark.parametrize("bad", [float("nan"), float("inf"), -float("inf")])
def test_non_finite_values_stay_in_their_channel_and_after(bad):
    import torch
    B, T, D = 2, 600, 66
    make, _ = problem(B, T, D, "float32", seed=6)
    x, r = make(B, T, D), make(B, T, D)
    rate = torch.from_numpy(chain_rates(D)).cuda()
    clean, _ = bstq.recur(x, r, rate)
    x[1, 333, 17] = bad
    h, hT = bstq.recur(x, r, rate)
    assert not torch.isfinite(h[1, 333:, 17]).any() and not torch.isfinite(hT[1, 17])
    h[1, 333:, 17], clean[1, 333:, 17] = 0, 0
    assert torch.equal(h, clean)


@pytest.mark.gpu
def test_equal_inputs_give_equal_bits():
    import torch
    B, T, D = 3, 3000, 200
    make, _ = problem(B, T, D, "bfloat16", seed=2)
    x, r, dh = make(B, T, D), make(B, T, D), make(B, T, D)
    rate = torch.from_numpy(chain_rates(D)).cuda()
    h, hT = bstq.recur(x, r, rate)
    first = bstq.recur_grad(x, r, rate, h, dh)
    for _ in range(5):
        h2, hT2 = bstq.recur(x, r, rate)
        assert torch.equal(h, h2) and torch.equal(hT, hT2)
        for u, v in zip(first, bstq.recur_grad(x, r, rate, h, dh)):
            assert torch.equal(u, v)


@pytest.mark.gpu
def test_many_sequences_share_one_rate_gradient():
    import torch
    B, T, D = 130, 65, 70
    make, _ = problem(B, T, D, "float32", seed=12)
    x, r, dh = make(B, T, D), make(B, T, D), make(B, T, D)
    rate = torch.from_numpy(chain_rates(D)).cuda()
    h, _ = bstq.recur(x, r, rate)
    got = bstq.recur_grad(x, r, rate, h, dh)
    check_gradients(got, reference_grad(f64(x), f64(r), f64(rate), f64(h), f64(dh)), f64(x), f64(h),
                    np.zeros((B, D)), T, "float32")


@pytest.mark.gpu
def test_offsets_past_32_bits():
    """A batch stride that takes the last sequence past 2^32 elements."""
    import torch
    T, D, far = 40, 64, (1 << 32) + 1024
    store = torch.empty(far + T * D, dtype=torch.bfloat16, device="cuda")
    x = store.as_strided((2, T, D), (far, D, 1))
    make, _ = problem(2, T, D, "bfloat16", seed=1)
    x.copy_(make(2, T, D))
    r = make(2, T, D)
    rate = torch.from_numpy(chain_rates(D)).cuda()
    h, hT = bstq.recur(x, r, rate)
    hd, hTd = bstq.recur(x.contiguous(), r, rate)
    assert torch.equal(h, hd) and torch.equal(hT, hTd)
    del store


@pytest.mark.gpu
def test_another_stream_and_a_given_workspace():
    import torch
    B, T, D = 2, 1500, 128
    make, _ = problem(B, T, D, "float32", seed=7)
    x, r = make(B, T, D), make(B, T, D)
    rate = torch.from_numpy(chain_rates(D)).cuda()
    want, last = bstq.recur(x, r, rate)
    nbytes = bstq.load().bstq_recur_work_size(bstq.F32, B, T, D)
    work = torch.full((nbytes,), 255, dtype=torch.uint8, device="cuda")
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    for _ in range(3):  # the workspace comes back as the last call left it
        h, hT = bstq.recur(x, r, rate, work=work, stream=side)
        side.synchronize()
        assert torch.equal(h, want) and torch.equal(hT, last)


@pytest.mark.gpu
def test_capture_in_a_graph():
    import torch
    B, T, D = 2, 900, 96
    make, _ = problem(B, T, D, "bfloat16", seed=7)
    x, r, dh = make(B, T, D), make(B, T, D), make(B, T, D)
    rate = torch.from_numpy(chain_rates(D)).cuda()
    bstq.recur_grad(x, r, rate, bstq.recur(x, r, rate)[0], dh)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        h, hT = bstq.recur(x, r, rate)
        grads = bstq.recur_grad(x, r, rate, h, dh)
    x.mul_(0.5)
    graph.replay()
    torch.cuda.synchronize()
    want, last = bstq.recur(x, r, rate)
    assert torch.equal(h, want) and torch.equal(hT, last)
    for u, v in zip(grads, bstq.recur_grad(x, r, rate, want, dh)):
        assert torch.equal(u, v)


# --------------------------------------------------------------------------
# One token
# --------------------------------------------------------------------------

@pytest.mark.gpu
@pytest.mark.parametrize("dtype", ["float32", "bfloat16", "float16"])
@pytest.mark.parametrize("B,D", [(1, 1), (1, 4096), (3, 33), (17, 258), (64, 1000)])
def test_one_token(B, D, dtype):
    import torch
    make, g = problem(B, 1, D, dtype, seed=B + D)
    x, r = make(B, 1, D)[:, 0], make(B, 1, D)[:, 0]
    rate = torch.from_numpy(chain_rates(D)).cuda()
    rows = 2 * B + 1
    state = torch.randn(rows, D, generator=g).cuda()
    slots = torch.randperm(rows, generator=g)[:B].to(torch.int32)
    if B > 2:
        slots[0], slots[1] = -1, rows  # two that take no part
    before = state.clone()
    h = bstq.recur_step(state, x, r, rate, slots=slots.cuda())
    used = [(b, int(s)) for b, s in enumerate(slots) if 0 <= s < rows]
    m = max(np.abs(f64(x)).max(), np.abs(f64(before)).max())
    want, last = reference(f64(x)[:, None], f64(r)[:, None], f64(rate),
                           f64(before)[[int(min(max(s, 0), rows - 1)) for s in slots]])
    for b, s in used:
        near(h[b], want[b, 0], 48 * U * m, dtype)
        near(state[s], last[b], 48 * U * m, "float32")
    idle = [s for s in range(rows) if s not in {s for _, s in used}]
    assert torch.equal(state[idle], before[idle])
    for b in range(B):
        if b not in {b for b, _ in used}:
            assert (h[b] == 0).all()
    state = before.clone()
    h = bstq.recur_step(state[:B], x, r, rate)
    want, last = reference(f64(x)[:, None], f64(r)[:, None], f64(rate), f64(before)[:B])
    near(h, want[:, 0], 48 * U * m, dtype)
    near(state[:B], last, 48 * U * m, "float32")
    assert torch.equal(state[B:], before[B:])


@pytest.mark.gpu
def test_tokens_one_by_one_follow_the_whole_sequence():
    import torch
    B, T, D = 3, 40, 130
    make, _ = problem(B, T, D, "float32", seed=21)
    x, r = make(B, T, D), make(B, T, D)
    rate = torch.from_numpy(chain_rates(D)).cuda()
    h, hT = bstq.recur(x, r, rate)
    _, state = bstq.recur(x[:, :25], r[:, :25], rate)
    wide = torch.zeros(B, D + 7, device="cuda")   # cache rows inside wider rows
    wide[:, :D] = state
    m = np.abs(f64(x)).max()
    for t in range(25, T):
        y = bstq.recur_step(wide[:, :D], x[:, t], r[:, t], rate)
        near(y, f64(h)[:, t], (64 + 16 * T ** 0.5) * U * m, "float32")
    near(wide[:, :D], f64(hT), (64 + 16 * T ** 0.5) * U * m, "float32")
    assert (wide[:, D:] == 0).all()


# --------------------------------------------------------------------------
# Empty axes and refusals
# --------------------------------------------------------------------------

@pytest.mark.gpu
def test_empty_axes():
    import torch
    rate = torch.ones(8, device="cuda")
    h0 = torch.randn(2, 8, device="cuda")
    x = torch.empty(2, 0, 8, device="cuda")
    h, hT = bstq.recur(x, x, rate, h0=h0)
    assert h.shape == (2, 0, 8) and torch.equal(hT, h0)
    dx, dr, drate, dh0 = bstq.recur_grad(x, x, rate, x, x, dhT=h0)
    assert dx.shape == (2, 0, 8) and (drate == 0).all() and torch.equal(dh0, h0)
    x = torch.empty(0, 5, 8, device="cuda")
    h, hT = bstq.recur(x, x, rate)
    assert h.shape == (0, 5, 8) and hT.shape == (0, 8)
    assert (bstq.recur_grad(x, x, rate, x, x)[2] == 0).all()
    x = torch.empty(2, 5, 0, device="cuda")
    assert bstq.recur(x, x, rate[:0])[0].shape == (2, 5, 0)
    assert bstq.recur_step(torch.empty(0, 8, device="cuda"), x[:0, 0, :].reshape(0, 0).new_empty(0, 8),
                           rate.new_empty(0, 8), rate).shape == (0, 8)


@pytest.mark.gpu
def test_refusals_of_the_binding():
    import torch
    x = torch.zeros(2, 5, 8, device="cuda")
    rate = torch.ones(8, device="cuda")
    good = dict(x=x, r=x, rate=rate)
    cases = [
        (TypeError, dict(x=x.double(), r=x.double())), (ValueError, dict(x=x[0], r=x[0])),
        (ValueError, dict(r=x[:, :4])), (ValueError, dict(r=x.bfloat16())), (ValueError, dict(x=x.cpu(), r=x.cpu())),
        (ValueError, dict(rate=rate[:7])), (ValueError, dict(rate=rate.double())), (ValueError, dict(rate=rate.cpu())),
        (ValueError, dict(h0=torch.zeros(2, 7, device="cuda"))), (ValueError, dict(h0=x[:, 0].bfloat16())),
        (ValueError, dict(lengths=torch.zeros(2, dtype=torch.int64, device="cuda"))),
        (ValueError, dict(x=torch.zeros(2, 5, 16, device="cuda")[:, :, ::2])),
        (ValueError, dict(out=x[:1])), (ValueError, dict(out=x[:1].expand(2, 5, 8))),
        (ValueError, dict(work=torch.zeros(8, dtype=torch.uint8, device="cuda"))),
    ]
    for kind, change in cases:
        with pytest.raises(kind):
            bstq.recur(**{**good, **change})
    for change in (dict(h=x[:, :4]), dict(dh=x.half()), dict(dhT=x[:, 0].half()), dict(h0=x[:, 0, :4])):
        with pytest.raises(ValueError):
            bstq.recur_grad(**{**good, "h": x, "dh": x, **change})
    s = torch.zeros(2, 8, device="cuda")
    for bad in (dict(state=s.half()), dict(state=s[:1]), dict(state=s[:, :7]), dict(r=s[:1]),
                dict(slots=torch.zeros(2, device="cuda")), dict(state=torch.zeros(8, 2, device="cuda").t())):
        with pytest.raises(ValueError):
            bstq.recur_step(**{"state": s, "x": s, "r": s, "rate": rate, **bad})


def _lib():
    import os
    if not os.path.exists(bstq.LIB_PATH):
        from symmetric_tridiagonal_eigensolver_gb300 import build
        build.build()
    return bstq.load()


def test_refusals_of_the_library():
    lib = _lib()
    buf = (ctypes.c_char * 4096)()
    base = ctypes.addressof(buf) + (-ctypes.addressof(buf)) % 256
    p = ctypes.c_void_p(base)
    odd = ctypes.c_void_p(base + 1)
    big = 1 << 31

    def codes(call, good, changes):
        for k, value, code in changes:
            args = list(good)
            args[k] = value
            assert call(*args) == code, (k, value)

    flat = (ctypes.c_int64 * 6)(40, 8, 40, 8, 40, 8)
    neg = (ctypes.c_int64 * 6)(40, -8, 40, 8, 40, 8)
    lap = (ctypes.c_int64 * 6)(40, 8, 40, 8, 40, 7)
    good = [0, 2, 5, 8, p, p, p, p, p, p, p, flat, p, None]
    codes(lib.bstq_recur, good, [
        (0, 1, -1), (0, 4, -1), (1, -1, -2), (1, big, -2), (2, -1, -3), (3, -1, -4), (3, big, -4), (4, None, -5),
        (4, odd, -5), (5, None, -6), (6, None, -7), (6, odd, -7), (7, odd, -8), (8, odd, -9), (9, None, -10),
        (10, odd, -11), (11, neg, -12), (11, lap, -12), (12, None, -13), (12, odd, -13), (1, 0, 0), (3, 0, 0)])
    assert lib.bstq_recur(0, 1 << 20, 1 << 20, 1 << 10, *good[4:]) == -4
    flat = (ctypes.c_int64 * 12)(*([40, 8] * 6))
    lap = (ctypes.c_int64 * 12)(*([40, 8] * 5 + [7, 8]))
    good = [0, 2, 5, 8, p, p, p, p, p, p, p, p, p, p, p, p, flat, p, None]
    codes(lib.bstq_recur_grad, good, [
        (0, 1, -1), (1, -1, -2), (2, -1, -3), (3, -1, -4), (4, None, -5), (5, odd, -6), (6, None, -7), (7, None, -8),
        (8, None, -9), (9, odd, -10), (10, odd, -11), (11, odd, -12), (12, None, -13), (13, odd, -14), (14, None, -15),
        (15, odd, -16), (16, lap, -17), (17, None, -18), (3, 0, 0)])
    three = (ctypes.c_int64 * 3)(8, 8, 7)
    good = [0, 2, 8, 2, p, 8, p, p, p, p, p, None, None]
    codes(lib.bstq_recur_step, good, [
        (0, 1, -1), (1, -1, -2), (2, -1, -3), (3, -1, -4), (4, None, -5), (4, odd, -5), (5, 7, -6), (6, None, -7),
        (7, odd, -8), (8, None, -9), (9, odd, -10), (10, None, -11), (11, three, -12), (1, 0, 0), (2, 0, 0)])
    good[9], good[3] = None, 1  # without slots the cache holds a row for each sequence
    assert lib.bstq_recur_step(*good) == -4
    for size in (lib.bstq_recur_work_size, lib.bstq_recur_grad_work_size):
        assert size(1, 2, 5, 8) == 0 and size(0, -1, 5, 8) == 0 and size(0, 2, 5, big) == 0
        assert size(0, 2, 5, 8) >= 256 and size(2, 2, 0, 8) >= 256
    import torch
    if not torch.cuda.is_available():
        assert lib.bstq_recur(0, 2, 5, 8, p, p, p, p, p, p, p, None, p, None) == bstq.ERR_NODEVICE


# --------------------------------------------------------------------------
# Gradients where a gate or a decay saturates, element by element
# --------------------------------------------------------------------------

def own_size(x, r, rate, h, dh, dhT, h0):
    """Gradients in 64 bits of sums without cancellation (dh, dhT, x - h >= 0) and
    a bound on each element's relative error, counted in u = 2^-24.

    The exponential of y = r log2 e has y's rounding, |r| u, and 4 u of its own;
    the gate s, and 1 - s, (|r| + 8) u; z = lambda s (|r| + 9) u, so a = exp(-z)
    is off by z (|r| + 9) u, by z u of its own y, and by 8 u.  A product of decays
    has the sum of theirs.  A sum of positive terms is off by at most the mean of
    what its terms are off by, weighted with them, and a rounding for each term."""
    B, T, D = x.shape
    s = 1 / (1 + np.exp(-r))
    o = 1 / (1 + np.exp(r))  # 1 - s
    lam = np.maximum(rate, 0)
    z = lam * s
    a, q = np.exp(-z), -np.expm1(-z)
    gate = np.abs(r) + 8
    off = z * (gate + 2) + 8
    dx, dr, ds = np.zeros_like(x), np.zeros_like(x), np.zeros_like(x)
    bx, br, bs = np.zeros_like(x), np.zeros_like(x), np.zeros_like(x)
    g, bg = dhT.astype(np.float64).copy(), np.zeros((B, D))
    for t in range(T - 1, -1, -1):
        before = h[:, t - 1] if t else h0
        new = g + dh[:, t]
        bg = np.where(new > 0, g * bg / np.where(new > 0, new, 1), bg) + 3
        g = new
        dx[:, t] = q[:, t] * g
        bx[:, t] = bg + gate[:, t] + 8
        g = a[:, t] * g
        bg = bg + off[:, t]
        ds[:, t] = g * (x[:, t] - before) * s[:, t]
        bs[:, t] = bg + gate[:, t] + 4
        dr[:, t] = ds[:, t] * lam * o[:, t]
        br[:, t] = bs[:, t] + gate[:, t] + 4
    drate = ds.sum((0, 1))
    brate = (ds * bs).sum((0, 1)) / np.maximum(drate, 1e-300) + 32 + 2 * (B * T) ** 0.5
    return (dx, dr, drate, g), (bx, br, brate, bg)


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", ["float32", "bfloat16"])
@pytest.mark.parametrize("T", [1, 6, 90, 400, 1500])
@pytest.mark.parametrize("kind", ["large rates", "open gates", "shut gates", "last token only"])
def test_gradients_keep_their_digits_where_gates_saturate(kind, T, dtype):
    """Rates of 8 to 30 and gates at up to |r| = 20: a = exp(-z) down to 1e-13 and
    1 - s down to 2e-9 are factors of dr, drate and dh0, which have to be right
    relative to their own size."""
    import torch
    B, D = 2, 70
    g = torch.Generator().manual_seed(T)

    def positive(*shape):
        return (torch.rand(*shape, generator=g) + 0.5).to(getattr(torch, dtype)).cuda()

    x, h, dh = positive(B, T, D), -positive(B, T, D), positive(B, T, D)
    lo, hi = {"large rates": (-3, 3), "open gates": (8, 20), "shut gates": (-20, -8), "last token only": (-3, 3)}[kind]
    r = (lo + (hi - lo) * torch.rand(B, T, D, generator=g)).to(x.dtype).cuda()
    top = {"large rates": 30.0, "open gates": 30.0, "shut gates": 1e4, "last token only": 6.0}[kind]
    rate = torch.linspace(0.2 * top, top, D).cuda()
    h0, dhT = -positive(B, D).float(), positive(B, D).float()
    if kind == "last token only":
        dh.zero_()
    got = bstq.recur_grad(x, r, rate, h, dh, dhT=dhT, h0=h0)
    want, bound = own_size(f64(x), f64(r), f64(rate), f64(h), f64(dh), f64(dhT), f64(h0))
    for name, v, w, b, kind_of in zip(("dx", "dr", "drate", "dh0"), got, want, bound, (dtype, dtype, "float32", "float32")):
        seen = w > 1e-30  # what 32 bits hold with room for the factors on the way
        err = np.abs(f64(v) - w)[seen] / w[seen]
        lim = b[seen] * U + HALF[kind_of]
        assert (err <= lim).all(), (name, (err / lim).max())


@pytest.mark.gpu
def test_gradients_of_saturated_gates_against_differences():
    """The loss sum(h dh) of the 64-bit recurrence, its slope along rate and r by
    central differences with steps relative to what they change."""
    import torch
    B, T, D = 1, 12, 8
    make, g = problem(B, T, D, "float32", seed=3)
    x, dh = make(B, T, D), make(B, T, D)
    r = make(B, T, D, shift=12.0)
    rate = torch.linspace(9.0, 16.0, D).cuda()
    h, _ = bstq.recur(x, r, rate)
    _, dr, drate, _ = bstq.recur_grad(x, r, rate, h, dh)
    base = [f64(x), f64(r), f64(rate)]

    def loss(p, j):  # of channel j, less what does not depend on rate and r: h_t = x_t + a_t (h_{t-1} - x_t)
        xx, rr, lam = p[0][0, :, j], p[1][0, :, j], p[2][j]
        last, out = 0.0, 0.0
        for t in range(T):
            rest = np.exp(-lam / (1 + np.exp(-rr[t]))) * (last - xx[t])
            out += rest * f64(dh)[0, t, j]
            last = xx[t] + rest
        return out

    for j in range(D):
        up, down = [v.copy() for v in base], [v.copy() for v in base]
        up[2][j] += 1e-4
        down[2][j] -= 1e-4
        slope = (loss(up, j) - loss(down, j)) / 2e-4
        # h enters as stored, rounded to 2^-24 of its size, which 1e-6 covers
        assert abs(float(drate[j]) - slope) <= 1e-4 * abs(slope) + 1e-6 * np.exp(-base[2][j]) * T


def test_outputs_whose_rows_overlap_are_refused():
    """An output's two strides have to keep all its rows apart, not only the
    neighbours along one axis: rows that two tiles write would race."""
    lib = _lib()
    import torch
    buf = (ctypes.c_char * 4096)()
    p = ctypes.c_void_p(ctypes.addressof(buf) + (-ctypes.addressof(buf)) % 256)

    def overlap(rows, n0, s0, n1, s1):
        at = sorted(i * s0 + j * s1 for i in range(n0) for j in range(n1))
        return any(b - a < rows for a, b in zip(at, at[1:]))

    rng = np.random.default_rng(0)
    layouts = [(2, 5, 8, 8, 8), (2, 5, 16, 8, 8), (2, 5, 40, 8, 8), (2, 5, 39, 8, 8), (2, 5, 8, 16, 8), (2, 5, 8, 15, 8),
               (2, 3, 6, 4, 2), (3, 2, 4, 6, 2), (2, 3, 7, 4, 2), (1, 5, 0, 8, 8), (2, 1, 8, 0, 8), (4, 4, 30, 10, 8)]
    layouts += [tuple(int(v) for v in rng.integers(1, [6, 6, 40, 40, 9])) for _ in range(300)]
    some = 0
    for batch, time, sb, st, dim in layouts:
        bad = overlap(dim, batch, sb, time, st)
        some += not bad
        if not bad and torch.cuda.is_available():
            continue  # these pointers are no device memory
        want = -12 if bad else bstq.ERR_NODEVICE
        dense = [time * dim, dim]
        assert lib.bstq_recur(0, batch, time, dim, p, p, p, None, None, p, None,
                              (ctypes.c_int64 * 6)(*dense, *dense, sb, st), p, None) == want, (batch, time, sb, st, dim)
        for k in (4, 5):
            strides = dense * 6
            strides[2 * k:2 * k + 2] = sb, st
            assert lib.bstq_recur_grad(0, batch, time, dim, p, p, p, p, p, None, None, None, p, p, p, None,
                                       (ctypes.c_int64 * 12)(*strides), p, None) == (-17 if bad else want)
    assert 20 < some < len(layouts) - 20
    far = 1 << 42  # no overflow on the way
    wide = (ctypes.c_int64 * 6)(40, 8, 40, 8, far, far - 3)
    assert lib.bstq_recur(0, 1 << 9, 1 << 9, 8, p, p, p, None, None, p, None, wide, p, None) == -12


@pytest.mark.gpu
def test_a_workspace_with_gaps_or_repeats_is_refused():
    """An expanded tensor counts more elements than its memory has."""
    import torch
    x = torch.zeros(2, 900, 64, device="cuda")
    rate = torch.ones(64, device="cuda")
    G = torch.zeros(200, 300, device="cuda")
    one = torch.zeros(1, dtype=torch.uint8, device="cuda")
    for work in (one.expand(1 << 28), torch.zeros(1 << 28, 2, dtype=torch.uint8, device="cuda")[:, 0]):
        for call in (lambda: bstq.recur(x, x, rate, work=work), lambda: bstq.recur_grad(x, x, rate, x, x, work=work),
                     lambda: bstq.orthogonalize(G, work=work)):
            with pytest.raises(ValueError, match="contiguous"):
                call()


def test_no_token_is_no_overlap():
    """A call without tokens has no rows, whatever its strides."""
    lib = _lib()
    import torch
    if torch.cuda.is_available():
        pytest.skip("the pointers are no device memory")
    buf = (ctypes.c_char * 4096)()
    p = ctypes.c_void_p(ctypes.addressof(buf) + (-ctypes.addressof(buf)) % 256)
    for strides in (None, (ctypes.c_int64 * 6)(*([0, 0] * 3))):
        assert lib.bstq_recur(0, 2, 0, 8, None, None, p, None, None, None, p, strides, p, None) == bstq.ERR_NODEVICE
    assert lib.bstq_recur_grad(0, 2, 0, 8, None, None, p, None, None, None, None, None, None, None, p, p, None, p,
                               None) == bstq.ERR_NODEVICE


# --------------------------------------------------------------------------
# A context with a part of the device's SMs
# --------------------------------------------------------------------------

class _Resource(ctypes.Structure):  # CUdevResource of an SM resource
    _fields_ = [("type", ctypes.c_int), ("padding", ctypes.c_ubyte * 92), ("sms", ctypes.c_uint),
                ("rest", ctypes.c_ubyte * 44)]


_green = []  # streams that tensors have been used on live as long as the process


def stream_on_a_part(sms):
    """A stream of a green context with some `sms` SMs; skips where the driver makes
    none."""
    import torch
    if not _green:
        cu = ctypes.CDLL("libcuda.so.1")
        whole, part, rest = _Resource(), _Resource(), _Resource()
        count, desc, ctx, handle = ctypes.c_uint(1), ctypes.c_void_p(), ctypes.c_void_p(), ctypes.c_void_p()
        ref = ctypes.byref
        torch.zeros(1, device="cuda")  # the primary context
        for call, args in ((cu.cuDeviceGetDevResource, (0, ref(whole), 1)),
                           (cu.cuDevSmResourceSplitByCount, (ref(part), ref(count), ref(whole), ref(rest), 0, sms)),
                           (cu.cuDevResourceGenerateDesc, (ref(desc), ref(part), 1)),
                           (cu.cuGreenCtxCreate, (ref(ctx), desc, 0, 1)),
                           (cu.cuGreenCtxStreamCreate, (ref(handle), ctx, 1, 0))):
            if call(*args) != 0:
                pytest.skip("no green contexts here")
        assert sms <= part.sms < whole.sms
        _green.extend((ctx, torch.cuda.ExternalStream(handle.value)))
    return _green[1]


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", ["float32", "bfloat16"])
@pytest.mark.parametrize("B,T,D", [(1, 9000, 64), (2, 3000, 1024)])
def test_a_context_with_a_part_of_the_sms(B, T, D, dtype):
    """Tiles wait for each other, so the grid has to fit the stream's own SMs."""
    import torch
    make, g = problem(B, T, D, dtype, seed=4)
    x, r, dh = make(B, T, D), make(B, T, D), make(B, T, D)
    rate = torch.from_numpy(chain_rates(D)).cuda()
    want = bstq.recur(x, r, rate)
    grads = bstq.recur_grad(x, r, rate, want[0], dh)
    torch.cuda.synchronize()
    stream = stream_on_a_part(16)
    got = bstq.recur(x, r, rate, stream=stream)
    mine = bstq.recur_grad(x, r, rate, want[0], dh, stream=stream)
    stream.synchronize()
    # the same tiles joined in other groups: roundings of the states, and of the type
    m = max(float(x.abs().max()), 1.0)
    near(got[0], f64(want[0]), (64 + 16 * T ** 0.5) * U * m, dtype)
    near(got[1], f64(want[1]), (64 + 16 * T ** 0.5) * U * m, "float32")
    for u, v, kind in zip(mine, grads, (dtype, dtype, "float32", "float32")):
        top = float(v.abs().max())
        near(u, f64(v), (64 + 16 * (B * T) ** 0.5) * U * 4 * top, kind)


# --------------------------------------------------------------------------
# Waits that run out
# --------------------------------------------------------------------------

def nan_or_equal(got, want):
    import torch
    return bool((torch.isnan(got) | (got == want)).all())


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", ["float32", "bfloat16"])
@pytest.mark.parametrize("B,T,D", [(1, 20000, 64), (1, 9000, 70), (6, 2500, 1024), (3, 700, 10000)])
def test_a_wait_that_runs_out_leaves_no_wrong_numbers(B, T, D, dtype):
    """With no cycles to wait, tiles give up on what the others have not published
    yet: the status says so, and every output is right or NaN."""
    import torch
    lib = bstq.load()
    make, g = problem(B, T, D, dtype, seed=1)
    x, r, dh = make(B, T, D), make(B, T, D), make(B, T, D)
    rate = torch.from_numpy(chain_rates(D)).cuda() + 0.01
    h0 = torch.randn(B, D, generator=g).cuda()
    lengths = torch.tensor([T - 7 * b for b in range(B)], dtype=torch.int32, device="cuda")
    kw = dict(h0=h0, lengths=lengths)
    want = bstq.recur(x, r, rate, **kw)
    grads = bstq.recur_grad(x, r, rate, want[0], dh, **kw)
    code = {"float32": bstq.F32, "bfloat16": bstq.BF16}[dtype]
    work = torch.zeros(max(lib.bstq_recur_work_size(code, B, T, D), lib.bstq_recur_grad_work_size(code, B, T, D)),
                       dtype=torch.uint8, device="cuda")
    status = work[:4].view(torch.int32)
    torch.cuda.synchronize()
    before = lib.bstq_set_wait_limit(0)
    try:
        for call, right in ((lambda: bstq.recur(x, r, rate, work=work, **kw), want),
                            (lambda: bstq.recur_grad(x, r, rate, want[0], dh, work=work, **kw), grads)):
            outs = call()
            torch.cuda.synchronize()
            gave_up = int(status)
            assert all(nan_or_equal(u, v) for u, v in zip(outs, right))
            missing = any(bool(torch.isnan(u).any()) for u in outs)
            assert gave_up == 1 and missing
    finally:
        assert lib.bstq_set_wait_limit(before) == 0
    again = bstq.recur(x, r, rate, work=work, **kw)
    assert int(status) == 0 and all(torch.equal(u, v) for u, v in zip(again, want))
    again = bstq.recur_grad(x, r, rate, want[0], dh, work=work, **kw)
    assert int(status) == 0 and all(torch.equal(u, v) for u, v in zip(again, grads))


def test_the_wait_limit_is_kept_and_given_back():
    lib = _lib()
    default = lib.bstq_set_wait_limit(7)
    assert default == 4000000000
    assert lib.bstq_set_wait_limit(-1) == 7
    assert lib.bstq_set_wait_limit(0) == default and lib.bstq_set_wait_limit(-5) == 0
