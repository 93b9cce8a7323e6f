"""Choices that fp32 scores cannot make: keys next to one another with exact ties among them."""
import pytest
import torch

import around_ref as A
from gpu_util import ensure_lib
from test_gpu_select import check, run

pytestmark = pytest.mark.gpu

FNS = ["softmax", "sqrt_softplus", "sigmoid"]


@pytest.fixture(scope="module")
def M():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    return ensure_lib()


def test_a_key_behind_a_tie_at_the_border(M):
    """sigmoid(20) and sigmoid(21) are one fp32 number, two equal experts of the former come first."""
    for E in (4, 8, 60, 256):
        for first in ([20.0, 20.0, 21.0], [20.0, 20.0, 20.0, 21.0], [20.0, 21.0, 20.0]):
            l = torch.full((1, E), -3.0)
            l[0, :len(first)] = torch.tensor(first)
            for K in (1, 2, 3):
                check(M, l, torch.zeros(E), K, "sigmoid")
                if E % 4 == 0 and K <= E // 4:
                    check(M, l, torch.zeros(E), K, "sigmoid", G=4, KG=1)


@pytest.mark.parametrize("fn", FNS)
@pytest.mark.parametrize("E", [8, 16, 31, 64, 100, 256])
def test_equal_experts_and_one_near_them(M, fn, E):
    """All experts are alike but one, whose bias brings its key next to theirs: by about a bias' last place, 1e-9, above or
    below, far less than fp32 tells apart.  (Where fp32 finds it below, it comes behind a tie at the border.)"""
    g = torch.Generator().manual_seed(E)
    told = 0
    for _ in range(16):
        l = torch.full((1, E), float(torch.randn(1, generator=g)))
        at = int(torch.randint(0, E, (1,), generator=g))
        l[0, at] = float(torch.randn(1, generator=g))
        s = A.score(l, fn)[0]
        bias = torch.full((E,), 0.1)
        other = (at + 1) % E
        bias[at] = float(s[other] + bias[other].double() - s[at])
        key = s + bias.double()
        if abs(float(key[at] - key[other])) < 1e-13:
            continue                     # 64-bit evaluations, good to 1e-15, have to tell them apart
        told += 1
        for K in (1, 2, 5):
            check(M, l.expand(3, E).contiguous(), bias, K, fn)
            if E % 8 == 0 and K <= E // 8 * 2:
                check(M, l, bias, K, fn, G=8, KG=2)
                check(M, l, bias, K, fn, G=8, KG=2, best=1)
    assert told >= 8


@pytest.mark.parametrize("fn", FNS)
def test_groups_whose_sum_fp32_cannot_hold(M, fn):
    """Two biases of fp32's lowest (or near its highest) value: their sum overflows in fp32, not in 64 bits, and such a group
    is worth more than one of -infinity."""
    low, inf = torch.finfo(torch.float32).min, float("inf")
    l = torch.randn(9, 32, generator=torch.Generator().manual_seed(7))
    for worst, mid in ((-inf, low), (-inf, 0.75 * low), (low, 0.875 * low), (-0.75 * low, -0.875 * low), (-inf, -low)):
        b = torch.randn(8, 4, generator=torch.Generator().manual_seed(8)) * 0.1
        b[0], b[1], b[4], b[6] = worst, worst, mid, mid
        for KG in (1, 2, 3, 5, 6, 7):
            for best in (1, 2):
                check(M, l, b.reshape(-1), 3, fn, G=8, KG=KG, best=best)


@pytest.mark.parametrize("bad", [float("nan"), float("inf")])
@pytest.mark.parametrize("E,G,KG,K,best", [(16, 4, 1, 3, 2), (16, 4, 2, 5, 1), (96, 12, 3, 8, 2), (256, 8, 4, 8, 2), (384, 12, 1, 10, 2)])
def test_softmax_rows_without_a_sum(M, bad, E, G, KG, K, best):
    """A NaN or infinite logit leaves a softmax row no sum: every score is NaN (a key of -infinity) but a masked expert's, which
    is 0 under every score function.  Groups go by that, experts without a bias by their logits."""
    g = torch.Generator().manual_seed(E + K)
    inf = float("inf")
    l = torch.randn(80, E, generator=g)
    l[torch.rand(80, E, generator=g) < torch.linspace(0, 0.9, 80)[:, None]] = -inf
    l[torch.arange(80), torch.randint(0, E, (80,), generator=g)] = bad
    ids, w = run(M, l, None, K, "softmax", G=G, KG=KG, best=best)
    n = E // G
    for t in range(80):
        key = [0.0 if v == -inf else -inf for v in l[t].tolist()]
        order = [-inf if v != v else v for v in l[t].tolist()]
        worth = [sum(sorted(key[i * n:(i + 1) * n], reverse=True)[:best]) for i in range(G)]
        groups = sorted(range(G), key=lambda i: (-worth[i], i))[:KG]
        allowed = [e for i in groups for e in range(i * n, (i + 1) * n)]
        assert ids[t].tolist() == sorted(allowed, key=lambda e: (-order[e], e))[:K], t
    # and two biases of fp32's lowest value in such a row
    low = torch.full((E,), torch.finfo(torch.float32).min)
    low[:n] = -inf
    l[:, n:2 * n] = -inf
    ids, _ = run(M, l, low, min(K, n), "softmax", G=G, KG=1, best=best)
    assert (ids >= n).all()
