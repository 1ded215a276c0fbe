"""The AdamW step over lists of tensors. Its rounding is defined (every operation
rounded to fp32 by itself, in the documented order), so with 32-bit states the
results are compared bit for bit with the same operations in numpy's fp32, and
those with the fp64 oracle: about ten roundings, 16 * 2^-24 of the parts. 8-bit
states are compared code by code with torch's e4m3 cast of the values. There the
root and the quotient are approximations of 2 ulp each: 2^-21 of the step, and a
root's code may be the other neighbour where the value is that close to halfway."""
import math

import numpy as np
import pytest
import torch

import oracle.tune_oracle as ot

pytestmark = pytest.mark.gpu
F = np.float32
HYPER = dict(lr=1e-2, betas=(0.9, 0.97), eps=1e-8, weight_decay=0.1, step=3)


@pytest.fixture(scope="module")
def kdkl():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from lm_head_top_gb300 import kdkl as m
    m.load()
    return m


def _bf16(x):
    return torch.from_numpy(x).bfloat16().float().numpy()


def _e4m3(x):
    return torch.from_numpy(x).to(torch.float8_e4m3fn).float().numpy()


def _quantise(x, keep_nonzero):
    """(values in units of their block's scale, scales) as the header defines the state."""
    n = x.size
    pad = np.zeros(-(-n // 256) * 256, dtype=F)
    pad[:n] = x
    blocks = pad.reshape(-1, 256)
    q, scales = np.zeros_like(blocks), np.ones(len(blocks), dtype=F)
    for i, b in enumerate(blocks):
        fin = np.abs(b[np.isfinite(b)])
        top = fin.max() if fin.size else F(0)
        if top > 0:
            half, e = np.frexp(top)
            scales[i] = F(2.0) ** max(int(e) - 9 + int(half > F(0.904383)), -126)
        y = b / scales[i]
        ok = np.isfinite(b)
        q[i] = np.where(ok, _e4m3(np.where(ok, y, 0).astype(F)), np.nan)
        if keep_nonzero:
            q[i] = np.where((y > 0) & (q[i] == 0), F(2.0 ** -9), q[i])
    return q.reshape(-1)[:n], scales


def _step(p, g, m, v, decay, lr, betas, eps, weight_decay, step, grad_scale=1.0):
    """fp32, operation by operation."""
    with np.errstate(all="ignore"):
        g = g * F(grad_scale)
        m = m * F(betas[0]) + g * F(1 - betas[0])
        v = v * F(betas[1]) + g * g * F(1 - betas[1])
        root = np.sqrt(v)
        den = root * F(1 / math.sqrt(1 - betas[1] ** step)) + F(eps)
        if decay:
            p = p * F(1 - lr * weight_decay)
        return p - m / den * F(lr / (1 - betas[0] ** step)), m, v, root


def _make(n, seed, state8, p16, g16):
    r = np.random.default_rng(seed)
    p = (r.normal(size=n) * 0.05).astype(F)
    g = (r.normal(size=n) * 1e-3 * 10.0 ** r.uniform(-3, 1, n)).astype(F)
    m, root = (r.normal(size=n) * 1e-3).astype(F), (r.random(n) * 1e-3).astype(F)
    p, g = (_bf16(p) if p16 else p), (_bf16(g) if g16 else g)
    if state8:
        return p, g, _quantise(m, False), _quantise(root, True)
    return p, g, m, root * root


def _dev(x, dtype, offset=0):
    t = torch.zeros(x.size + offset, dtype=dtype, device="cuda")[offset:]
    t.copy_(torch.from_numpy(x).to(dtype))
    return t


def _near(got, want, off):
    ok = np.isfinite(want)
    assert np.array_equal(np.isfinite(got), ok)
    assert (np.abs(got - want) <= off)[ok].all()


def _run(kdkl, sizes, state8=False, p16=False, g16=False, copy=True, offset=0, decay=None,
         mutate=None, **hyper):
    h = {**HYPER, **hyper}
    data = [_make(n, 10 * i + n % 7, state8, p16, g16) for i, n in enumerate(sizes)]
    if mutate:
        mutate(data)
    pt, gt = (torch.bfloat16 if p16 else torch.float32), (torch.bfloat16 if g16 else torch.float32)
    params = [_dev(d[0], pt, offset) for d in data]
    grads = [_dev(d[1], gt, offset) for d in data]
    copies = [torch.zeros(n + offset, dtype=torch.bfloat16, device="cuda")[offset:] for n in sizes] \
        if copy else None
    if state8:
        m = [_dev(d[2][0], torch.float8_e4m3fn, offset) for d in data]
        v = [_dev(d[3][0], torch.float8_e4m3fn, offset) for d in data]
        ms, vs = [_dev(d[2][1], torch.float32) for d in data], \
            [_dev(d[3][1], torch.float32) for d in data]
    else:
        m, v = [_dev(d[2], torch.float32, offset) for d in data], \
            [_dev(d[3], torch.float32, offset) for d in data]
        ms = vs = None
    handle = kdkl.kd_adamw_tensors(params, grads, m, v, copies=copies, m_scales=ms, v_scales=vs,
                                   decay=decay)
    kdkl.kd_adamw_step(handle, **h)
    torch.cuda.synchronize()
    np32 = lambda t: t.float().cpu().numpy()  # noqa: E731
    for i, (p, g, a, b) in enumerate(data):
        if state8:
            scale = lambda s, n: np.repeat(s, 256)[:n]  # noqa: E731
            n = p.size
            a = a[0] * scale(a[1], n)
            b = (b[0] * scale(b[1], n)) ** 2
        step = {k: h[k] for k in ("lr", "betas", "eps", "weight_decay", "step")}
        want_p, want_m, want_v, root = _step(p, g, a, b, decay is None or decay[i],
                                             grad_scale=h.get("grad_scale", 1.0), **step)
        if state8:
            with np.errstate(all="ignore"):
                off = np.abs(want_p - p) * F(2.0 ** -21) + np.abs(want_p) * F(2.0 ** -23)
            _near(np32(params[i]), want_p, off + (np.abs(want_p) * F(2.0 ** -8) if p16 else 0))
            if copy:
                _near(np32(copies[i]), want_p, off + np.abs(want_p) * F(2.0 ** -8))
            q, s = _quantise(want_m, False)
            assert np.array_equal(np32(m[i]), q, equal_nan=True), i
            assert np.array_equal(np32(ms[i]), s), i
            q, s = _quantise(root, True)
            assert np.array_equal(np32(vs[i]), s), i
            got, y = np32(v[i]), root / np.repeat(s, 256)[:p.size]
            ok = np.isfinite(q)
            assert np.array_equal(np.isnan(got), ~ok) and np.array_equal(got > 0, q > 0), i
            assert (np.abs(got - y) <= np.abs(q - y) + y * F(2.0 ** -20))[ok].all(), i
        else:
            assert np.array_equal(np32(params[i]), _bf16(want_p) if p16 else want_p,
                                  equal_nan=True), i
            if copy:
                assert np.array_equal(np32(copies[i]), _bf16(want_p), equal_nan=True), i
            assert np.array_equal(np32(m[i]), want_m, equal_nan=True), i
            assert np.array_equal(np32(v[i]), want_v, equal_nan=True), i
    return data, params


SIZES = [1, 7, 8, 255, 256, 257, 2048, 0, 8191, 8192, 8193, 100003]


@pytest.mark.parametrize("state8", [False, True])
@pytest.mark.parametrize("p16", [False, True])
@pytest.mark.parametrize("g16", [False, True])
def test_types_and_sizes(kdkl, state8, p16, g16):
    _run(kdkl, SIZES, state8, p16, g16, copy=not p16)


@pytest.mark.parametrize("state8", [False, True])
def test_unaligned_views(kdkl, state8):
    _run(kdkl, SIZES, state8, offset=1)
    _run(kdkl, SIZES, state8, g16=True, offset=3)


@pytest.mark.parametrize("count", [32, 33, 384, 385, 800])
def test_many_tensors(kdkl, count):
    before = kdkl.kd_launch_count()
    _run(kdkl, [1 + (37 * i) % 300 for i in range(count)],
         decay=[i % 3 != 0 for i in range(count)])
    assert kdkl.kd_launch_count() - before == -(-count // 384)


def test_many_blocks_and_scales(kdkl):
    for state8 in (False, True):
        _run(kdkl, [1 << 20, 3, (1 << 18) + 77], state8, grad_scale=0.25, eps=1e-6, step=1000)


@pytest.mark.parametrize("n", [7_000_003, 13_000_300])
def test_8bit_blocks_of_several_passes(kdkl, n):
    """Enough elements for thread blocks that make 2 and 4 passes."""
    _run(kdkl, [n, 5, 4097], True, g16=True)


def test_device_scale(kdkl):
    n = 1000
    out = []
    for kw in (dict(grad_scale=0.5), dict(grad_scale=2.0, grad_scale_dev=torch.full((1,), 0.25,
                                                                                  device="cuda"))):
        p, g, m, v = (_dev(x, torch.float32) for x in _make(n, 0, False, False, False))
        kdkl.kd_adamw_step(kdkl.kd_adamw_tensors([p], [g], [m], [v]), **HYPER, **kw)
        out.append((p, m, v))
    assert all(torch.equal(a, b) for a, b in zip(*out))


@pytest.mark.parametrize("state8", [False, True])
def test_first_step_and_zero_gradients(kdkl, state8):
    def zero(data):
        for i, (p, g, a, b) in enumerate(data):
            if state8:
                data[i] = (p, g, (np.zeros_like(a[0]), np.ones_like(a[1])),
                           (np.zeros_like(b[0]), np.ones_like(b[1])))
            else:
                data[i] = (p, g, np.zeros_like(a), np.zeros_like(b))
        data[1][1][:] = 0  # a tensor whose gradient is zero: nothing but decay
    data, params = _run(kdkl, [600, 600, 5000], state8, mutate=zero, step=1)
    assert np.array_equal(params[1].cpu().numpy(), data[1][0] * F(1 - 1e-3))  # 0 / eps is exact


@pytest.mark.parametrize("state8", [False, True])
def test_infinities_and_nan_stay_where_they_are(kdkl, state8):
    def spoil(data):
        data[0][1][5], data[0][1][300], data[0][1][301] = np.nan, np.inf, -np.inf
    _, params = _run(kdkl, [1000, 1000], state8, mutate=spoil)
    bad = ~torch.isfinite(params[0])
    assert bad.nonzero().squeeze(1).tolist() == [5, 300, 301]
    assert torch.isfinite(params[1]).all()


def test_tiny_values(kdkl):
    """Gradients whose squares vanish, blocks below the smallest scale."""
    def tiny(data):
        for p, g, a, b in data:
            g *= F(1e-36)
    _run(kdkl, [700], False, mutate=tiny)
    def tiny8(data):
        p, g, a, b = data[0]
        data[0] = (p, g * F(1e-30), (a[0] * 0, a[1]), (b[0] * 0, b[1]))
    _run(kdkl, [700], True, mutate=tiny8)


def test_against_fp64(kdkl):
    n = 4096
    p, g, m, v = _make(n, 1, False, False, False)
    got = [_dev(x, torch.float32) for x in (p, g, m, v)]
    kdkl.kd_adamw_step(kdkl.kd_adamw_tensors([got[0]], [got[1]], [got[2]], [got[3]]), **HYPER,
                       grad_scale=0.5)
    want = ot.adamw(*(x.astype(np.float64) for x in (p, g, m, v)), **HYPER, grad_scale=0.5)
    parts = (np.abs(p) + np.abs(want[0] - p),
             np.abs(m) + np.abs(g), np.abs(want[2]))
    for t, w, part in zip((got[0], got[2], got[3]), want, parts):
        # a cancelling m also scales its step: that error is the second part of p's bound
        assert (np.abs(t.cpu().numpy() - w) <= 16 * 2.0 ** -24 * (part + 1e-2) ).all()


def test_8bit_states_train(kdkl):
    """A least-squares fit reaches the same loss with 8-bit states as with 32-bit ones."""
    torch.manual_seed(0)
    A, y = torch.randn(512, 300, device="cuda"), torch.randn(512, device="cuda")
    best = ((A @ torch.linalg.lstsq(A, y).solution - y) ** 2).mean().item()
    ends = []
    for state8 in (False, True):
        p, g = torch.zeros(300, device="cuda"), torch.zeros(300, device="cuda")
        dt = torch.float8_e4m3fn if state8 else torch.float32
        m, v = torch.zeros(300, device="cuda").to(dt), torch.zeros(300, device="cuda").to(dt)
        ones = [torch.ones(2, device="cuda") for _ in range(2)]
        h = kdkl.kd_adamw_tensors([p], [g], [m], [v], m_scales=[ones[0]] if state8 else None,
                                  v_scales=[ones[1]] if state8 else None)
        for i in range(400):
            g.copy_(2 * A.t() @ (A @ p - y) / 512)
            kdkl.kd_adamw_step(h, lr=1e-2 if i < 300 else 1e-3, step=i + 1)
        ends.append(((A @ p - y) ** 2).mean().item())
    assert ends[0] <= 1.05 * best and ends[1] <= 1.1 * best
