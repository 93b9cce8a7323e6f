"""Rows whose elements lie past 2^31 (and bytes past 2^32) from the first one's."""
import pytest
import torch

from gpu_util import ensure_lib

pytestmark = pytest.mark.gpu

BF = torch.bfloat16
T, H = 320000, 7168            # 2.29e9 elements


@pytest.fixture(scope="module")
def M():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    if torch.cuda.get_device_properties(0).total_memory < 64 << 30:
        pytest.skip("needs 64 GB")
    return ensure_lib()


def block(n, c, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    return torch.randn(n, c, generator=g, device="cuda")


def far(n, c, dt, seed, base=1000):
    """n rows of a block of 1000 in turn (a row 2^31 or 2^32 elements or bytes away is another of them)."""
    b = block(base, c, seed).to(dt)
    return b.repeat(n // base, 1)


def near_and_far(n):
    return [0, 1, n // 2 + 3, n - 1001, n - 2, n - 1]


def test_norm_and_gradients(M):
    x, w, eps = far(T, H, BF, 1), torch.rand(H, device="cuda") + 0.5, 1e-5
    y, x8 = torch.empty_like(x), M.new_rows8(T, H)
    M.rms_norm(x, w, eps, y=y, y8=x8)
    ref, ref8 = torch.empty(1000, H, dtype=BF, device="cuda"), M.new_rows8(1000, H)
    M.rms_norm(x[:1000], w, eps, y=ref, y8=ref8)
    rows = near_and_far(T)
    small = [r % 1000 for r in rows]
    # (their sums may be taken in another order: two roundings of bf16 at most)
    assert ((y[rows].float() - ref[small].float()).abs() <= 2.0 ** -7 * ref[small].float().abs()).all()
    assert torch.equal(x8[1][rows], ref8[1][small]) and (x8[0][rows].int() - ref8[0][small].int()).abs().max() <= 1
    del x8
    dy, ws = far(T, H, BF, 2), M.new_workspace_norm(T, H)
    M.rms_norm_backward(dy, x, w, eps, y, ws)
    M.rms_norm_backward(dy[:1000], x[:1000], w, eps, ref, M.new_workspace_norm(1000, H))
    size = ref[small].float().abs().amax(1, keepdim=True)
    assert ((y[rows].float() - ref[small].float()).abs() <= 2.0 ** -7 * ref[small].float().abs() + 2.0 ** -16 * size).all()
    assert M.get_error(ws) == M.OK


def test_8_bit_rows(M):
    x = far(T, H, BF, 3)
    x8, out = M.new_rows8(T, H), torch.empty_like(x)
    M.pack_rows8(x, x8)
    small = M.new_rows8(1000, H)
    M.pack_rows8(x[:1000], small)
    rows = near_and_far(T)
    at = [r % 1000 for r in rows]
    assert torch.equal(x8[0][rows], small[0][at]) and torch.equal(x8[1][rows], small[1][at])
    M.unpack_rows8(x8, out)
    ref = torch.empty(1000, H, dtype=BF, device="cuda")
    M.unpack_rows8(small, ref)
    assert torch.equal(out[rows], ref[at])
    # through an index that reads from the far end first
    ids, ws = torch.arange(T - 1, -1, -1, dtype=torch.int32, device="cuda"), torch.zeros(256, dtype=torch.uint8, device="cuda")
    M.unpack_rows8(x8, out, x_ids=ids, ws=ws)
    assert torch.equal(out[rows], ref[[(T - 1 - r) % 1000 for r in rows]]) and M.get_error(ws) == M.OK


def test_routing(M):
    n, E, K = 9000000, 256, 2
    l = far(n, E, torch.float32, 4)
    ids, w = torch.empty(n, K, dtype=torch.int32, device="cuda"), torch.empty(n, K, device="cuda")
    M.select(l, ids, w, "sigmoid", n_groups=8, topk_groups=2)
    small = torch.empty(1000, K, dtype=torch.int32, device="cuda"), torch.empty(1000, K, device="cuda")
    M.select(l[:1000], *small, "sigmoid", n_groups=8, topk_groups=2)
    rows = near_and_far(n)
    at = [r % 1000 for r in rows]
    assert torch.equal(ids[rows], small[0][at]) and torch.equal(w[rows], small[1][at])
    assert torch.equal(ids.view(-1, 1000, K), small[0].expand(n // 1000, 1000, K))
    ws = M.new_workspace_rows(n, K, E)
    out, ref = torch.empty(n, E, dtype=BF, device="cuda"), torch.empty(1000, E, dtype=BF, device="cuda")
    M.select_backward(l, ids, w, w, out, ws, "sigmoid")
    M.select_backward(l[:1000], *small, small[1], ref, ws, "sigmoid")
    assert torch.equal(out[rows], ref[at]) and M.get_error(ws) == M.OK
