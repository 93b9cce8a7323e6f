"""Activation gradients of experts' rows without a bias gradient, whose CTAs walk over all experts' rows, against the pass with
one, which goes expert by expert: the same bits, however the rows are spread over the experts."""
import pytest
import torch

import train_ref as R
from gpu_util import ensure_lib

pytestmark = pytest.mark.gpu

BF, HF = torch.bfloat16, torch.float16


@pytest.fixture(scope="module")
def M():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    return ensure_lib()


def spread(kind, E, total):
    """Counts of E experts, `total` rows in all or about."""
    if kind == "even":
        return [total // E + (e < total % E) for e in range(E)]
    if kind == "one":
        return [total if e == E // 2 else 0 for e in range(E)]
    if kind == "halves":
        return [int(total * 0.5 ** (e + 1)) for e in range(E)]
    if kind == "last":
        return [0] * (E - 1) + [total]
    g = torch.Generator().manual_seed(E)
    share = torch.softmax(torch.randn(E, generator=g) * 2, 0)
    return torch.bincount(torch.multinomial(share, total, True, generator=g), minlength=E).tolist()


def both(M, dt, act, counts, align, N, rows, seed=0, K=16):
    """(dx, status) of the call without and with a bias gradient."""
    E, g = len(counts), torch.Generator(device="cuda").manual_seed(seed)
    cols = N // 2 if act == "swiglu" else N
    dy = torch.randn(rows, cols, generator=g, device="cuda").to(dt)
    z = torch.randn(rows, N, generator=g, device="cuda").to(dt)
    w = torch.randn(E, N, K, generator=g, device="cuda").to(dt) * 0.1
    c = torch.tensor(counts, dtype=torch.int32, device="cuda")
    out = []
    for bias in (False, True):
        ws = M.new_workspace_linear(rows, N, K, E, act)
        dx = torch.full((rows, K), 7.25, dtype=dt, device="cuda")
        db = torch.empty(E, N, device="cuda") if bias else None
        M.linear_backward(dy, None, w, ws, dx=dx, dbias=db, act=act, z=z, expert_counts=c, align=align)
        out.append((dx, M.get_error(ws)))
    return dy, z, w, out


@pytest.mark.parametrize("kind", ["even", "one", "halves", "last", "random"])
@pytest.mark.parametrize("E,total,align,N", [(1, 300, 1, 48), (3, 700, 16, 528), (32, 5000, 16, 256), (64, 640, 64, 80), (257, 900, 1, 128),
                                             (300, 40, 4, 1040), (1024, 3000, 2, 32), (1024, 1024, 16, 16), (8, 20000, 16, 2048)])
def test_rows_spread_over_experts(M, kind, E, total, align, N):
    counts = spread(kind, E, total)
    rows = sum(-(-n // align) * align for n in counts) + 5
    for dt in (BF, HF):
        for act in ("relu", "silu", "gelu", "swiglu"):
            dy, z, w, ((a, sa), (b, sb)) = both(M, dt, act, counts, align, N, rows)
            assert sa == sb == M.OK
            assert torch.equal(a, b), (act, dt)
    # and by the formula, for the last of them
    for e, r, n in R.segments(counts, align, rows)[:: max(1, E // 8)]:
        if n:
            s = slice(r, r + n)
            (dx, ex), _, _ = R.linear_grad(dy[s].cpu(), torch.zeros(n, 16, dtype=dt), w[e].cpu(), z[s].cpu(), act, None, dt)
            R.check(a[s], dx, ex, "dx")


@pytest.mark.parametrize("counts", [[4, 100, 3], [-1, 4, 6], [2147483647, 2147483647, 1], [5, -7, 100], [0, 0, 33], [32, 1, 1]])
def test_counts_that_leave_the_buffers(M, counts):
    """They are cut to the buffers and reported, by either pass."""
    for align in (1, 16):
        _, _, _, ((a, sa), (b, sb)) = both(M, BF, "silu", counts, align, 64, 32)
        assert sa == sb == M.ERR_DEVICE_INDEX
        assert torch.equal(a, b)


def test_buffers_wider_than_the_rows(M):
    """Rows that are likely there are told by the buffers' size; more or fewer of them change nothing."""
    for rows in (64, 100, 5000, 40000):
        for counts in ([40, 0, 3], [0, 0, 0], [1, 1, 1]):
            _, _, _, ((a, sa), (b, sb)) = both(M, BF, "gelu", counts, 16, 272, rows)
            assert sa == sb == M.OK and torch.equal(a, b)
