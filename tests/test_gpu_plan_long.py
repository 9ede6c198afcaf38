"""Sorts of long batches: on both sides of the size from which the chunks' histograms get a launch of their own, and
their time, which grows with the slots and not with their square."""
import numpy as np
import pytest
import torch

import moe_grouped_gemm_02_amd as fg
from fgtest import dev, to_dev
from test_gpu_rows import host, plan_ids

pytestmark = pytest.mark.gpu


def reference(ids, G, start):
    """Each slot's (expert or G, rank) by a stable sort, and its row from the experts' first rows."""
    flat = ids.reshape(-1).astype(np.int64)
    key = np.where((flat >= 0) & (flat < G), flat, G)
    order = np.argsort(key, kind="stable")
    counts = np.bincount(key, minlength=G + 1)
    first = start(counts[:G])
    rank = np.empty(flat.size, np.int64)
    rank[order] = np.arange(flat.size) - np.repeat(np.cumsum(counts) - counts, counts)
    return key, rank, np.append(first, 0)[key] + rank, counts[:G], first


@pytest.mark.parametrize("kind", ["random", "wild", "one", "none", "sorted"])
@pytest.mark.parametrize("T,k,G,align,M_max", [(8192, 8, 256, 128, 300), (8449, 8, 256, 16, 300), (4099, 8, 1024, 64, 20),
                                               (30011, 8, 64, 128, 4000), (70000, 8, 7, 1, 9000), (150001, 8, 300, 128, 4096),
                                               (310000, 7, 1024, 16, 2000)])
def test_long_plans(T, k, G, align, M_max, kind):
    print(f"plan {T}x{k} G={G} align={align} M_max={M_max} {kind}", flush=True)
    ids = plan_ids(kind, T, k, G, T + G)
    p = fg.plan_contiguous(to_dev(ids), G, align)
    ends = lambda n: np.cumsum(-(-n // align) * align)  # noqa: E731
    key, rank, row, counts, first = reference(ids, G, lambda n: ends(n) - -(-n // align) * align)
    there = key < G
    slots, m = np.full(p.capacity, -1), np.full(p.capacity, -1)
    slots[row[there]], m[row[there]] = np.flatnonzero(there), key[there]
    assert np.array_equal(host(p.offsets), np.append(first, ends(counts)[-1]))
    assert np.array_equal(host(p.rows).reshape(-1), np.where(there, row, -1))
    assert np.array_equal(host(p.slots), slots) and np.array_equal(host(p.m_indices), m)
    p = fg.plan_masked(to_dev(ids), G, M_max)
    there &= rank < M_max
    row = key * M_max + rank
    slots = np.full(G * M_max, -1)
    slots[row[there]] = np.flatnonzero(there)
    assert np.array_equal(host(p.masked_m), np.minimum(counts, M_max))
    assert np.array_equal(host(p.rows).reshape(-1), np.where(there, row, -1)) and np.array_equal(host(p.slots), slots)


def test_long_plan_in_a_graph():
    ids = to_dev(plan_ids("random", 40000, 8, 200, 3))
    fg.plan_contiguous(ids, 200)
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        p = fg.plan_contiguous(ids, 200)
    for r in range(4):
        ids.copy_(ids.flip(0))
        want = fg.plan_contiguous(ids, 200)
        torch.cuda.synchronize()
        g.replay()
        torch.cuda.synchronize()
        assert torch.equal(p.rows, want.rows) and torch.equal(p.slots, want.slots) and torch.equal(p.offsets, want.offsets)
        assert torch.equal(p.m_indices, want.m_indices)


def test_time_grows_with_the_slots():
    """Four times the slots: about three times the time (with every histogram summed by every workgroup it was 13)."""
    best = []
    for slots in (1 << 20, 1 << 22):
        ids = torch.randint(0, 1024, (slots // 8, 8), dtype=torch.int32, device=dev())
        fg.plan_contiguous(ids, 1024)
        times = []
        for _ in range(8):
            a, b = torch.cuda.Event(enable_timing=True), torch.cuda.Event(enable_timing=True)
            a.record()
            fg.plan_contiguous(ids, 1024)
            b.record()
            torch.cuda.synchronize()
            times.append(a.elapsed_time(b))
        best.append(min(times))
    print(best, flush=True)
    assert best[1] <= 7 * best[0]
