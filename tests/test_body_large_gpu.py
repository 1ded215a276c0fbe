"""The embedding and the norms where counts and offsets are large: sorts beyond a quarter of a
million tokens, and arrays of more than 2^31 elements, whose last rows lie past 32 bits."""
import pytest
import torch

from oracle import body_oracle as bo

pytestmark = pytest.mark.gpu
U = 2.0 ** -24


@pytest.fixture(scope="module")
def kdkl():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from lm_head_top_gb300 import kdkl as m
    m.load()
    return m


@pytest.fixture(autouse=True)
def memory_is_given_back():
    yield
    torch.cuda.empty_cache()


def _gen(seed):
    return torch.Generator("cuda").manual_seed(seed)


@pytest.mark.parametrize("T", [262_144, 262_145, 300_001, 1_000_003])
@pytest.mark.parametrize("V", [1000, 700_000])
@pytest.mark.parametrize("accumulate", [False, True])
def test_sorts_of_many_tokens(kdkl, T, V, accumulate):
    """Tiles grow beyond 1024 tokens from 262,145 on."""
    d, g = 8, _gen(T)
    ids = (V * torch.rand(T, generator=g, device="cuda") ** 2).int().clamp_(max=V - 1)
    ids[torch.rand(T, generator=g, device="cuda") < 0.02] = V // 3
    mask = (torch.rand(T, generator=g, device="cuda") < 0.8).to(torch.uint8)
    dY = torch.randn(T, d, generator=g, device="cuda")
    dW = torch.randn(V, d, generator=g, device="cuda") if accumulate else None
    want, size, count = bo.embedding_backward(dY, ids, V, mask, 0.3, dW)
    dY[mask == 0] = float("nan")
    ws = torch.full((kdkl.kd_embedding_workspace_size(T, d, V, 1),), 0xFF, dtype=torch.uint8, device="cuda")
    if accumulate:
        got = kdkl.kd_embedding_backward(dY, ids, mask, scale=0.3, dW=dW, accumulate_dW=True, workspace=ws)
    else:
        got = kdkl.kd_embedding_backward(dY, ids, mask, scale=0.3, dW=torch.full((V, d), float("nan"), device="cuda"), workspace=ws)
    assert kdkl.kd_kl_check_status(ws) == 0
    # a piece's 31 sums at most, its pieces' one after the other, the scale, its product, the last sum
    chain = count.clamp(max=31) + count / 32 + 5
    assert ((got.double() - want).abs() <= chain[:, None] * U * 1.01 * size).all()
    if not accumulate:
        assert torch.equal(got, kdkl.kd_embedding_backward(dY, ids, mask, scale=0.3, V=V))


@pytest.mark.parametrize("d", [2880, 2877])
def test_rows_of_a_table_past_32_bits(kdkl, d):
    V, T = 750_000, 333
    assert V * d > 2 ** 31
    W = torch.empty(V, d, dtype=torch.bfloat16, device="cuda")
    W[-400:].normal_(generator=_gen(1))
    W[:400].normal_(generator=_gen(2))
    ids = torch.cat([torch.arange(V - 200, V), torch.arange(T - 200)]).int().cuda()
    got = kdkl.kd_embedding_forward(W, ids, scale=2.0)
    assert torch.equal(got, W[ids.long()] * 2)
    dY = torch.randn(T, d, generator=_gen(3), device="cuda")
    dW = kdkl.kd_embedding_backward(dY, ids, V=V)
    assert torch.equal(dW[ids.long()], dY) and not dW[T - 200:V - 200].any()
    kdkl.kd_embedding_backward(dY, ids, dW=dW, accumulate_dW=True)
    assert torch.equal(dW[ids.long()], 2 * dY) and not dW[T - 200:V - 200].any()


@pytest.mark.parametrize("d", [2880, 2877])
def test_tokens_past_32_bits(kdkl, d):
    T, V = 750_000, 1000
    W = torch.randn(V, d, generator=_gen(4), device="cuda").bfloat16()
    ids = (torch.arange(T, device="cuda") % (V - 3)).int()
    ids[-3:] = torch.arange(V - 3, V, device="cuda").int()  # theirs alone
    Y = kdkl.kd_embedding_forward(W, ids)
    for at in (0, T // 2, T - 1000):
        assert torch.equal(Y[at:at + 1000], W[ids[at:at + 1000].long()])
    # the gradient of rows that are the table's: n times each, as powers of two hold it
    Y.copy_(torch.where(Y < 0, -1.0, 1.0))
    dW = kdkl.kd_embedding_backward(Y, ids, V=V)
    count = torch.bincount(ids.long(), minlength=V).float()
    assert torch.equal(dW, torch.where(W < 0, -1.0, 1.0) * count[:, None])


@pytest.mark.parametrize("kind,d", [("rms", 2880), ("layer", 2877)])
def test_norms_of_rows_past_32_bits(kdkl, kind, d):
    T, layer = 750_000, kind == "layer"
    assert T * d > 2 ** 31
    g = _gen(5)
    x, r = (torch.empty(T, d, dtype=torch.bfloat16, device="cuda").normal_(generator=g) for _ in range(2))
    w, b = torch.randn(d, generator=g, device="cuda"), torch.randn(d, generator=g, device="cuda") if layer else None
    y, h, mean, rstd = kdkl.kd_norm_forward(x, w, b, residual=r, kind=kind)
    parts = [slice(at, at + 500) for at in (0, T // 2, T - 500)]
    row = 64 * U  # of a sum over a row
    for s in parts:
        wy, wh, wmean, wrstd = bo.norm(x[s], w, b, r[s], kind)
        off = row * wh.double().abs().mean(1) if layer else torch.zeros_like(wrstd)
        rel = row + (off * wrstd) ** 2 + 2 * U
        assert torch.equal(h[s], wh) and ((rstd[s].double() - wrstd).abs() <= rel * wrstd).all()
        size = ((wh.double() - wmean[:, None]).abs() * (rel + 4 * U)[:, None] + off[:, None]) * wrstd[:, None] * w.double().abs()
        if layer:
            size = size + U * (wy.abs() + b.double().abs())
        assert ((y[s].double() - wy).abs() <= size + 2.0 ** -8 * 1.01 * (wy.abs() + size)).all()
    dx, dw, db = kdkl.kd_norm_backward(r, h, w, mean, rstd, dh=x, kind=kind, want_dbias=layer, dx=y)
    for s in parts:
        m = mean[s] if layer else None
        wx = bo.norm_backward(r[s], h[s], w, m, rstd[s], x[s], kind)[0]
        n = (h[s].double() - (m.double()[:, None] if layer else 0)).abs() * rstd[s].double()[:, None]
        k = r[s].double().abs() * w.double().abs()
        size = row * rstd[s].double()[:, None] * (k + n * (k * n).mean(1, keepdim=True) + k.mean(1, keepdim=True))
        size = size + U * (wx.abs() + x[s].double().abs())
        assert ((dx[s].double() - wx).abs() <= size + 2.0 ** -8 * 1.01 * (wx.abs() + size)).all()
    # the sums over all rows, in parts
    sums = torch.zeros(4, d, dtype=torch.double, device="cuda")
    for at in range(0, T, 50_000):
        s = slice(at, at + 50_000)
        n = (h[s].double() - (mean[s].double()[:, None] if layer else 0)) * rstd[s].double()[:, None]
        dy = r[s].double()
        sums += torch.stack([(dy * n).sum(0), (dy * n).abs().sum(0), dy.sum(0), dy.abs().sum(0)])
    # a block's rows one after the other (two blocks an SM or more), the blocks' by 32, then 32 in order
    chain = (-(-T // 304) + 8 + 16 * 152 // 32 + 32 + 8) * U
    assert ((dw.double() - sums[0]).abs() <= chain * sums[1]).all()
    if layer:
        assert ((db.double() - sums[2]).abs() <= chain * sums[3]).all()
