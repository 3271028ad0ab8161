"""dA and dB of the backward from an 8-bit checkpoint to 24 bits of their fp32 factor:
s v and s u enter the matrix units in three bf16 parts (8 bits each), and none may be
missing or in another's place.

Tolerances.  What is left is fp32: a sum of M products in chains of at most M / 32
instructions and a few slices, each off by at most (M / 32 + 32) 2^-24 of the sum of
their magnitudes (v itself, a sum over `rows`, likewise); over all elements errors of
random sign, 2^-24 sqrt(M / 32 + rows / 32) of that sum's own size, below 1e-6 of the
result at the sizes below.  Two parts alone leave 2^-17 of the factor: 2e-6 and more."""
import pytest
import torch

from tests._gpu import needs_gpu, say
from tests.test_gpu_act8 import _case, _ref, _rel, qn  # noqa: F401

pytestmark = [pytest.mark.gpu, needs_gpu]
TOL = 1e-6

# every rank block, dropout, rows that end inside steps and slices, calls whose slices
# are added by their own launch and by a tile's last workgroup
CASES = [(31, 72, 192, 5, 0.0), (33, 520, 576, 17, 0.0), (100, 136, 1024, 32, 0.1),
         (300, 520, 576, 33, 0.0), (129, 1024, 640, 48, 0.05), (1000, 264, 320, 64, 0.3),
         (2048, 1024, 1024, 16, 0.0), (4096, 512, 2048, 8, 0.05), (4100, 2056, 2112, 16, 0.0),
         (2500, 1032, 1088, 40, 0.05)]


@pytest.mark.parametrize("M,rows,cols,r,p", CASES)
def test_three_parts(qn, M, rows, cols, r, p):  # noqa: F811
    say(f"[act8 parts] M={M} rows={rows} cols={cols} r={r} p={p}")
    st, x, A, B, G, mask = _case(qn, M, rows, cols, r, p, seed=M + r)
    x8, alpha = qn.act8_pack(x), 2.0 * r
    u = torch.randn(M, r, generator=torch.Generator().manual_seed(r)).cuda()
    _, dA, dB = qn.qlora_linear_bwd_act8(st, x8, G, A, B, alpha, u, need_dx=False,
                                         dropout_mask=mask, dropout_p=p)
    torch.cuda.synchronize()
    _, dA64, dB64 = _ref(qn, st, x8, A, B, G, u, alpha / r / (1 - p), mask)
    say(f"    dA {_rel(dA, dA64):.2e} dB {_rel(dB, dB64):.2e}")
    assert _rel(dA, dA64) <= TOL and _rel(dB, dB64) <= TOL


@pytest.mark.parametrize("M,rows,cols,r", [(64, 64, 128, 3), (96, 72, 192, 16), (128, 136, 320, 33),
                                           (256, 64, 64, 64), (4096, 64, 4096, 16)])
def test_rows_that_cancel_leave_the_third_part(qn, M, rows, cols, r):  # noqa: F811
    """Rows in pairs m, m + 1 with opposite G and the same x: u of the second differs in
    its last bits only, so that dB is a sum of last bits: G^T of (u_m - u_m+1), which the
    first two parts hold none of.  The products of a pair cancel exactly whatever their
    order in fp32 (each is G times a part, eight bits by eight)."""
    say(f"[act8 cancel] M={M} rows={rows} cols={cols} r={r}")
    st, x, A, B, _, _ = _case(qn, M, rows, cols, r, 0.0, seed=M + r)
    g = torch.Generator().manual_seed(M)
    # G: one row of +-1 and its opposite a pair, one pair alone in each column
    G = torch.zeros(M, rows)
    for c in range(rows):
        m = 2 * (c * 7 % (M // 2))
        G[m, c], G[m + 1, c] = 1.0, -1.0
    # u: 1 + 2^-9 + 2^-18 a with a = 1 or 2 in the first row of a pair, 0 in the second: bf16
    # parts 1, 2^-9 and 2^-18 a
    u = torch.full((M, r), 1.0 + 2.0 ** -9)
    last = torch.randint(1, 3, (M // 2, r), generator=g).float() * 2.0 ** -18
    u[0::2] += last
    G16 = G.to(torch.bfloat16).cuda()
    _, _, dB = qn.qlora_linear_bwd_act8(st, qn.act8_pack(x), G16, A, B, float(r), u.cuda(),
                                        need_dx=False)
    torch.cuda.synchronize()
    want = G.double().t() @ u.double()
    assert want.abs().max() <= 2.0 ** -17 and want.abs().min() >= 2.0 ** -18
    assert torch.equal(dB.cpu().double(), want)


@pytest.mark.parametrize("M,rows,cols,r", [(64, 64, 128, 3), (96, 72, 192, 16), (128, 136, 320, 33),
                                           (256, 64, 64, 64), (4096, 64, 4096, 16)])
def test_the_third_part_of_v(qn, M, rows, cols, r):  # noqa: F811
    """The same for dA: v = G B of a pair is 1 + 2^-9 + 2^-18 a and -(1 + 2^-9), exactly, and
    x has one pair of equal ones in each column."""
    say(f"[act8 cancel v] M={M} rows={rows} cols={cols} r={r}")
    st, _, A, _, _, _ = _case(qn, M, rows, cols, r, 0.0, seed=M + r)
    g = torch.Generator().manual_seed(M + 1)
    a = torch.randint(1, 3, (M // 2,), generator=g).float() * 2.0 ** -18
    G = torch.zeros(M, rows)
    G[0::2, 0], G[0::2, 5], G[0::2, rows - 1] = 1.0, 2.0 ** -9, a
    G[1::2, 0], G[1::2, 5] = -1.0, -2.0 ** -9
    x = torch.zeros(M, cols)
    pair = torch.arange(cols) * 7 % (M // 2)
    x[2 * pair, torch.arange(cols)] = x[2 * pair + 1, torch.arange(cols)] = 1.0
    bf = lambda v: v.to(torch.bfloat16).cuda()  # noqa: E731
    _, dA, _ = qn.qlora_linear_bwd_act8(st, qn.act8_pack(bf(x)), bf(G), A,
                                        bf(torch.ones(rows, r)), float(r),
                                        torch.zeros(M, r, device="cuda"), need_dx=False)
    torch.cuda.synchronize()
    assert torch.equal(dA.cpu(), a[pair].expand(r, cols))
