"""The Muon step's arithmetic restated on the CPU: every matrix as two fp16 halves, products of
three, sums that lose towards zero with every 16 terms and are taken out every 8 blocks of 64. With
a part of it left out on request, to see what the tolerances of the tests on the GPU would notice."""
import torch

from oracle import body_oracle as bo

A, B, C = bo.QUINTIC
# What kd_muon_step may be off in X after 5 steps, in the 2-norm and relative to it: three times
# the 1e-5 that the header states. The restatement is 1e-6 to 3e-6 off at the tests' sizes (its sums
# lose less than the tensor core's), and with any one of the six smaller products left out 2e-4 or
# more.
X_TOL = 3e-5
# After one step of a matrix of rank one, whose products add up terms of one sign. A sum of up to
# 96 instructions loses half a unit of a running sum with each: of the sum itself, whose running
# value is half of it on average and whose unit 2^-23 to 2^-24 of it, 96 x 2^-23 / 2 / 2 x 0.75 =
# 2.1e-6. At a singular value of 1, where X becomes (3.4445 - 4.775 + 2.0315) X = 0.701 X, what S loses
# counts (4.775 - 2 x 2.0315) / 0.701 = 1.0 times, what S^2 loses 2.0315 / 0.701 = 2.9 times and
# what P X loses 2.7435 / 0.701 = 3.9 times: 1.6e-5, and a fifth more for the halves' own 2^-22.
# The restatement is 2.3e-6 off, and 8e-5 without the sums in registers at 20,000 columns.
X_TOL_ONE = 2e-5


def halves(x, scale):
    v = (x * scale).float()
    hi = v.half()
    return hi.double(), (v - hi.float()).half().double()


def _toward_zero(x):
    """To 24 bits."""
    return (x.contiguous().view(torch.int64) & ~((1 << 29) - 1)).view(torch.float64)


def _product(a, b, drop, blocks_a_sum):
    depth = a[0].shape[1]
    total = torch.zeros(a[0].shape[0], b[0].shape[1], dtype=torch.double)
    part = torch.zeros_like(total)
    blocks = -(-depth // 64)
    for block in range(blocks):
        for k in range(64 * block, min(depth, 64 * block + 64), 16):
            s = slice(k, min(depth, k + 16))
            for i, j in ((0, 0), (0, 1), (1, 0)):
                if drop != (i, j):
                    part = _toward_zero(part + a[i][:, s] @ b[j][s])
        if block + 1 == blocks or (block + 1) % blocks_a_sum == 0:
            total = (total + part).float().double()
            part = torch.zeros_like(total)
    return total


def x_of(u, steps=5, drop=None, blocks_a_sum=8):
    """X of u (rows <= columns). drop: (which of S, S^2 and P X, which of the halves' products)."""
    def left_out(which):
        return drop[1] if drop is not None and drop[0] == which else None
    u = u.float()
    X = halves(u / u.square().sum().sqrt(), 2.0 ** 13)
    for _ in range(steps):
        S = halves(_product(X, [x.t().contiguous() for x in X], left_out(0), blocks_a_sum) * 2.0 ** -13, 1.0)
        SS = _product(S, S, left_out(1), blocks_a_sum)
        P = halves(B * 2.0 ** -2 * (S[0] + S[1]) + C * 2.0 ** -15 * SS, 1.0)
        X = halves(A * (X[0] + X[1]) + 2.0 ** -11 * _product(P, X, left_out(2), blocks_a_sum), 1.0)
    return (X[0] + X[1]) * 2.0 ** -13


def rank_one(rows, cols, generator, device="cpu"):
    def side(n):
        r = torch.rand(2, n, generator=generator, device=device)
        return (0.5 + r[0]) * torch.where(r[1] < 0.5, -1.0, 1.0)
    return side(rows)[:, None] * side(cols)
