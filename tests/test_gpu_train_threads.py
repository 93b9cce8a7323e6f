"""Calls of several sizes from two host threads at once, each with a stream, a workspace and buffers of its own."""
import threading

import pytest
import torch

from gpu_util import ensure_lib

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def M():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    return ensure_lib()


class Dispatch:
    """One dispatch of T tokens of 8 columns; `call` repeats it, `outputs` are what it writes."""

    def __init__(self, M, T, E, K, align=4, H=8):
        self.M, self.E, self.align = M, E, align
        g = torch.Generator().manual_seed(T + E)
        self.ids = torch.rand(T, E, generator=g).topk(K, 1).indices.to(torch.int32).cuda()
        self.x = torch.randn(T, H, generator=g).cuda()
        U = M.msum_upper(T, K, E, align)
        self.x_perm = torch.zeros(U, H, device="cuda")
        self.sorted, self.experts = (torch.zeros(U, dtype=torch.int32, device="cuda") for _ in range(2))
        self.inv, self.m_sum = torch.zeros_like(self.ids), torch.zeros(1, dtype=torch.int32, device="cuda")
        self.ws = M.new_workspace_rows(T, K, E)

    def call(self):
        self.M.dispatch(self.ids, self.x, self.E, self.align, self.x_perm, self.sorted, self.experts, self.inv, self.m_sum,
                        self.ws)

    def outputs(self):
        return self.x_perm, self.sorted, self.experts, self.inv, self.m_sum


def together(jobs, calls):
    """Runs every job's call `calls` times, each job on a thread and a stream of its own: what they raised."""
    errors, start = [], threading.Barrier(len(jobs))

    def work(job):
        try:
            with torch.cuda.stream(torch.cuda.Stream()):
                start.wait()
                for _ in range(calls):
                    job.call()
        except Exception as e:      # noqa: BLE001 (any of them fails the test)
            errors.append(e)

    threads = [threading.Thread(target=work, args=(j,)) for j in jobs]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    torch.cuda.synchronize()
    return errors


def check_together(M, jobs, calls):
    want = []
    for j in jobs:
        j.call()
        want.append([t.clone() for t in j.outputs()])
        for t in j.outputs():
            t.zero_()
    torch.cuda.synchronize()
    assert together(jobs, calls) == []
    for j, w in zip(jobs, want):
        assert M.get_error(j.ws) == M.OK
        assert all(torch.equal(a, b) for a, b in zip(j.outputs(), w))


def test_dispatch_of_some_hundred_pairs(M):
    # index arrays in one launch, whose shared memory goes by pairs and experts: 78 KB and 2 KB
    check_together(M, [Dispatch(M, 340, 512, 6), Dispatch(M, 150, 8, 2)], 40000)


class Permute(Dispatch):
    """The layer's permute of as many pairs, without rows."""

    def __init__(self, M, T, E, K, align=4):
        super().__init__(M, T, E, K, align)
        self.ws = M.new_workspace(T, 128, 128, E, K, align)

    def call(self):
        self.M.permute(self.ids, self.E, self.align, self.sorted, self.experts, self.inv, self.m_sum, self.ws)

    def outputs(self):
        return self.sorted, self.experts, self.inv, self.m_sum


def test_dispatch_of_some_thousand_pairs(M):
    # index arrays by the layer's permute: 136 KB and 1 KB of shared memory
    check_together(M, [Dispatch(M, 2048, 1024, 2), Dispatch(M, 2048, 8, 2)], 40000)


def test_permute_of_some_hundred_pairs(M):
    # 8 KB and 64 bytes
    check_together(M, [Permute(M, 100, 1024, 6), Permute(M, 100, 8, 6)], 40000)
