"""The entry of a token's own id in the gradient of the logits, g (1 - p) / tau: in
fp32 from the token's logit and lse, never rounded to bf16, for confident tokens too.

Tolerances. The other entries, -g p_v / tau, are rounded to bf16 once (at most 2^-8
of each), an output in bf16 once more (2^-8 of it). The own entry is g/tau times
-expm1(logp), so it is off by g/tau times logp's error: half a step of lse (2^-24 of
it), a few fp32 roundings of the logit and of the sum of exponentials, some 2^-22 each.
64 * 2^-24 * max(1, |lse|, sum |h w| / tau / 8) holds them; 0.1 % of an entry is the
least that a rounding to bf16 would be told by, so entries above 16 times that are told.
For d = 2880, random rounding of 90 products a lane and of 32 lanes is some 1.6e-6 at
logits of 25, half a step of lse 1e-6, the forward's own error 1e-6: 1e-5 is 5 sigma."""
import pytest
import torch

pytestmark = pytest.mark.gpu
U16 = 2.0 ** -8
SLACK = 1 + 2.0 ** -6  # the bf16 rounding is taken of a value that is itself off


@pytest.fixture(scope="module")
def kdkl():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from lm_head_top_gb300 import kdkl as m
    m.load()
    return m


def _case(T, d, V, tau, ids, lean, seed=0):
    """H leans towards its token's row by `lean` [T]: the own logit is about lean / tau."""
    g = torch.Generator("cuda").manual_seed(seed)
    W = (torch.randn(V, d, generator=g, device="cuda") / d ** 0.5).bfloat16()
    H = (0.5 * torch.randn(T, d, generator=g, device="cuda")
         + lean[:, None] * W[ids.long()].float()).bfloat16()
    grad = torch.randn(T, generator=g, device="cuda")
    return H, W, grad


def _want(H, W, ids, grad, tau):
    """dH, dW, and the sums of the magnitudes of their terms that pass through bf16, in 64 bits."""
    Hd, Wd = H.double(), W.double()
    logs = torch.log_softmax(Hd @ Wd.t() / tau, 1)
    at = torch.arange(len(ids), device="cuda")
    p = logs.exp()
    slope = -p
    slope[at, ids.long()] = -torch.expm1(logs[at, ids.long()])
    p[at, ids.long()] = 0
    up = grad.double()[:, None] / tau
    slope = slope * up
    rest = (p * up).abs()
    return slope @ Wd, slope.t() @ Hd, rest @ Wd.abs(), rest.t() @ Hd.abs(), slope, logs


def _delta(H, W, ids, tau, logs):
    hw = (H.double() * W.double()[ids.long()]).abs().sum(1) / tau
    lse = (H.double() * W.double()[ids.long()]).sum(1) / tau - logs.gather(1, ids.long()[:, None])[:, 0]
    one = torch.ones_like(hw)
    return 64 * 2.0 ** -24 * torch.maximum(torch.maximum(one, lse.abs()), hw / 8)


def _run(kdkl, H, W, ids, grad, tau, **kw):
    _, lse = kdkl.kd_logprob_forward(H, W, ids, temperature=tau)
    return kdkl.kd_logprob_backward(H, W, ids, lse, grad, temperature=tau, **kw)


def _hold(got, want, rest, label, half_step):
    off = (got.double() - want).abs()
    room = U16 * SLACK * rest + label + (U16 * SLACK * want.abs() if half_step else 0) + 1e-9
    worst = (off / room).max().item()
    assert worst <= 1, worst


@pytest.mark.parametrize("tau", [1.0, 0.7])
def test_each_entry_to_fp32(kdkl, tau):
    """One token per id, a fp32 dW: what dW's row holds along the token's H."""
    T, d, V = 384, 64, 4096
    ids = torch.arange(0, 10 * T, 10, dtype=torch.int32, device="cuda")
    lean = torch.linspace(0, 18 * tau, T, device="cuda")
    H, W, grad = _case(T, d, V, tau, ids, lean)
    _, dW = _run(kdkl, H, W, ids, grad, tau)
    _, want, _, rest, slope, logs = _want(H, W, ids, grad, tau)
    Hd, rows = H.double(), ids.long()
    size = (Hd * Hd).sum(1)
    off = ((dW.double() - want)[rows] * Hd).sum(1).abs() / size
    room = (grad.double().abs() / tau * _delta(H, W, ids, tau, logs)
            + U16 * SLACK * (rest[rows] * Hd.abs()).sum(1) / size + 2.0 ** -20 * slope.gather(
                1, rows[:, None])[:, 0].abs())
    assert (off <= room).all(), (off / room).max().item()
    told = slope.gather(1, rows[:, None])[:, 0].abs() * 2.0 ** -9 > room
    assert told.sum().item() > T // 4  # enough of them would notice a rounding to bf16


@pytest.mark.parametrize("rest", [1e-2, 1e-3, 1e-4, 1e-5])
def test_confident_tokens(kdkl, rest):
    """1 - p down to 1e-5 at logits of 25 and d = 2880."""
    T, d, V = 64, 2880, 512
    g = torch.Generator("cuda").manual_seed(7)
    ids = torch.arange(0, 2 * T, 2, dtype=torch.int32, device="cuda")
    W = (torch.randn(V, d, generator=g, device="cuda") / d ** 0.5)
    # the own row and its neighbour: two logits that carry all of the mass
    H = 25 * W[ids.long()] / (W[ids.long()] ** 2).sum(1, keepdim=True)
    gap = torch.log(torch.tensor(1 / rest))
    W[ids.long() + 1] = (1 - gap / 25) * W[ids.long()]
    H, W = H.bfloat16(), W.bfloat16()
    grad = torch.ones(T, device="cuda")
    _, dW = _run(kdkl, H, W, ids, grad, 1.0)
    _, want, _, _, slope, _ = _want(H, W, ids, grad, 1.0)
    Hd, rows = H.double(), ids.long()
    size = (Hd * Hd).sum(1)
    got = (dW.double()[rows] * Hd).sum(1) / size
    exact = (want[rows] * Hd).sum(1) / size
    assert 0.3 * rest < slope.gather(1, rows[:, None]).mean().item() < 3 * rest
    assert ((got - exact).abs() <= 1e-5 + 2.0 ** -20 * exact).all(), ((got - exact).abs()).max().item()


SHAPES = [(1, 8, 2, 4096), (300, 72, 513, 4096), (300, 72, 513, 40), (700, 320, 2050, 4096),
          (700, 320, 2050, 100)]


@pytest.mark.parametrize("T,d,V,chunk", SHAPES)
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("spread", ["one", "few", "all"])
def test_every_element(kdkl, T, d, V, chunk, dtype, spread):
    """dH and dW element by element, ids of one, of a few and of all rows, so that a row
    of dW has one token's term or many."""
    tau = 0.8
    g = torch.Generator("cuda").manual_seed(T + V)
    u = torch.rand(T, generator=g, device="cuda")
    ids = {"one": 0 * u + (V - 1), "few": u * min(V, 5) * (V // 5 if V > 5 else 1), "all": u * V}[spread]
    ids = ids.int().clamp_(max=V - 1)
    H, W, grad = _case(T, d, V, tau, ids, 6 * torch.rand(T, generator=g, device="cuda"))
    grad[::7] = 0
    dH, dW = _run(kdkl, H, W, ids, grad, tau, dW_dtype=dtype, chunk=chunk)
    want_dH, want_dW, rest_dH, rest_dW, slope, logs = _want(H, W, ids, grad, tau)
    delta = grad.double().abs() / tau * _delta(H, W, ids, tau, logs) + 2.0 ** -20 * slope.abs().sum(1)
    rows = ids.long()
    label = torch.zeros_like(want_dW).index_add_(0, rows, delta[:, None] * H.double().abs())
    # fp32 sums of T terms and the accumulation of the products, block by block
    sums = 2.0 ** -20 * (slope.abs().t() @ H.double().abs())
    _hold(dW, want_dW, rest_dW, label + sums, dtype == torch.bfloat16)
    _hold(dH, want_dH, rest_dH, delta[:, None] * W.double()[rows].abs()
          + 2.0 ** -20 * (slope.abs() @ W.double().abs()), True)
    assert not dH[::7].any()


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
def test_repeated_ids_far_apart(kdkl, dtype):
    """5000 tokens: one id on every third, one twice at the ends, the others a few times;
    the same bits from run to run."""
    T, d, V, tau = 5000, 72, 900, 1.0
    g = torch.Generator("cuda").manual_seed(3)
    ids = (torch.rand(T, generator=g, device="cuda") * (V - 2)).int()
    ids[::3] = V - 1
    ids[1] = ids[T - 1] = V - 2
    H, W, grad = _case(T, d, V, tau, ids, 5 * torch.rand(T, generator=g, device="cuda"))
    dH, dW = _run(kdkl, H, W, ids, grad, tau, dW_dtype=dtype)
    want_dH, want_dW, rest_dH, rest_dW, slope, logs = _want(H, W, ids, grad, tau)
    delta = grad.double().abs() / tau * _delta(H, W, ids, tau, logs) + 2.0 ** -20 * slope.abs().sum(1)
    label = torch.zeros_like(want_dW).index_add_(0, ids.long(), delta[:, None] * H.double().abs())
    _hold(dW, want_dW, rest_dW, label + 2.0 ** -18 * (slope.abs().t() @ H.double().abs()),
          dtype == torch.bfloat16)
    _hold(dH, want_dH, rest_dH, delta[:, None] * W.double()[ids.long()].abs()
          + 2.0 ** -20 * (slope.abs() @ W.double().abs()), True)
    again = _run(kdkl, H, W, ids, grad, tau, dW_dtype=dtype)
    assert torch.equal(again[0], dH) and torch.equal(again[1], dW)


def test_own_entries_are_added_to_dW_once(kdkl):
    """Accumulated over two calls and over token and vocabulary blocks."""
    T, d, V = 600, 128, 1500
    g = torch.Generator("cuda").manual_seed(5)
    ids = (torch.rand(T, generator=g, device="cuda") * 40).int()
    H, W, grad = _case(T, d, V, 1.0, ids, torch.zeros(T, device="cuda"))
    _, want, _, rest, slope, logs = _want(H, W, ids, grad, 1.0)
    _, lse = kdkl.kd_logprob_forward(H, W, ids)
    dW = torch.zeros(V, d, device="cuda")
    for half in (slice(0, 250), slice(250, T)):
        kdkl.kd_logprob_backward(H[half], W, ids[half], lse[half], grad[half], dW=dW, chunk=40,
                                 accumulate_dW=True)
    delta = grad.double().abs() * _delta(H, W, ids, 1.0, logs)
    label = torch.zeros_like(want).index_add_(0, ids.long(), delta[:, None] * H.double().abs())
    _hold(dW, want, rest, label + 2.0 ** -18 * (slope.abs().t() @ H.double().abs()), False)
