"""Scratch of the packed scan, from its sizes alone (no GPU)."""
import pytest
import torch

import gated_deltanet_linear_18_b200 as gdn

BF, F32 = torch.bfloat16, torch.float32
RECORD = (2 * 128 * 5 + 16) * 4              # a chunk's decay vectors of 128 columns
MOST = 2 ** 31 - 1


@pytest.fixture(scope="module", autouse=True)
def built():
    from gated_deltanet_linear_18_b200 import _build
    _build.build()


def test_scratch_grows_with_the_rows_and_not_with_the_bound():
    f = gdn.ssm_scan_workspace_bytes
    # 512 requests under a bound of 16384, 64 heads of 64 in pairs: 20000 / 128 + 512 records a pair at most
    assert f(512, 16384, 64, 1, 64, 128, BF, total=20000) == 256 + 32 * (20000 // 128 + 512) * RECORD
    # three requests of 48 rows in all: the bound is cut at the rows
    for bound in (48, 49, 5000, MOST):
        assert f(3, bound, 2, 1, 64, 64, BF, total=48) == 256 + 3 * RECORD
    # where every sequence may be as long as its neighbours, no more than a record for each of their chunks
    assert f(4, 2048, 4, 1, 64, 128, BF, total=8192) == f(4, 2048, 4, 1, 64, 128, BF)


def test_scratch_of_a_packed_call_is_never_above_the_one_without_its_rows():
    f = gdn.ssm_scan_workspace_bytes
    for nseq in (1, 2, 7, 150, 3000):
        for bound in (1, 127, 128, 129, 1000, 40000):
            for total in (1, 128, 1000, 123457):
                for H, G, P, N in ((3, 1, 64, 128), (48, 16, 128, 128), (64, 1, 64, 64)):
                    assert 0 < f(nseq, bound, H, G, P, N, BF, total=total) <= f(nseq, bound, H, G, P, N, BF)


def test_no_scratch():
    f = gdn.ssm_scan_workspace_bytes
    assert f(3, 0, 2, 1, 64, 64, BF, total=5) == 0 and f(3, 5, 2, 1, 64, 64, BF, total=0) == 0
    assert f(3, 5, 2, 1, 64, 64, BF, total=-1) == 0 and f(3, 5, 2, 1, 64, 64, F32, total=5) == 0
    assert f(0, 5, 2, 1, 64, 64, BF, total=5) == 0 and f(3, 5, 2, 1, 32, 64, BF, total=5) == 0


def test_records_of_packed_sequences_are_their_own():
    """Sequence s has its chunks' records from (first row) / 128 + s on: none shared, none beyond rows / 128 + nseq."""
    g = torch.Generator().manual_seed(1)
    for _ in range(200):
        n = int(torch.randint(1, 40, (1,), generator=g))
        gaps, lens = (torch.randint(0, m, (n,), generator=g) * torch.randint(0, 2, (n,), generator=g) for m in (200, 700))
        at, used, total = 0, [], int(gaps.sum() + lens.sum())
        for s in range(n):
            at += int(gaps[s])
            used += range(at // 128 + s, at // 128 + s + max(-(-int(lens[s]) // 128), 1))
            at += int(lens[s])
        assert len(set(used)) == len(used) and max(used) < total // 128 + n
