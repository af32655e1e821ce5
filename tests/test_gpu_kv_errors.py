"""Errors of the KV-cache calls next to other work: a skipped index is reported, and nothing else
on the device takes notice of it."""
import time

import pytest
import torch

import kv_plain as P
from test_gpu_kv_cache import i32, rows, to_gpu

pytestmark = pytest.mark.gpu
ERR_WAIT_GRID, ERR_INDEX = 1 << 3, 1 << 4


@pytest.fixture(scope="module")
def dv():
    import mixed_precision_weight_b200 as pkg
    return pkg.binding


@pytest.fixture(autouse=True)
def no_device_error(dv):
    dv.dvssq_device_error(clear=True)
    yield
    assert dv.dvssq_device_error(clear=True) == 0


def test_a_bad_index_does_not_end_a_grid_wait_on_another_stream(dv):
    """A grid barrier gives up early when a kernel elsewhere gave up a wait.  A row that a KV-cache call
    skips is not that: the wait (of a counter that nothing increments) lasts its whole limit."""
    pool, table, _ = P.filled(1, 2, 128, [100], seed=1)
    c, k, past = to_gpu(dv, pool, table), rows(1, 2, 128, 2).cuda(), i32([64 * table.shape[1]])
    dv.dvssq_kv_append(c, k, k, past)
    assert dv.dvssq_device_error(clear=True) == ERR_INDEX
    cycles = 400_000_000
    dv.dvssq_set_wait_limit(cycles)
    try:
        s1, s2 = torch.cuda.Stream(), torch.cuda.Stream()
        a, b = torch.cuda.Event(enable_timing=True), torch.cuda.Event(enable_timing=True)
        torch.cuda.synchronize()
        a.record(s1)
        dv.dvssq_selftest_wait(1, stream=s1)
        b.record(s1)
        time.sleep(0.02)                                    # the wait has begun
        dv.dvssq_kv_append(c, k, k, past, stream=s2)
        torch.cuda.synchronize()
        ms = a.elapsed_time(b)
    finally:
        dv.dvssq_set_wait_limit(0)
    assert dv.dvssq_device_error(clear=True) == ERR_WAIT_GRID | ERR_INDEX
    assert ms > cycles / 2e9 * 1e3, ms                      # the limit at 2 GHz, above the clock's maximum


@pytest.mark.parametrize("d", [64, 256])
@pytest.mark.parametrize("start,n", [([-3, 5], [70, 4]), ([-64, 0], [65, 1]), ([-200, -1], [330, 66]), ([-5, -70], [5, 3])])
def test_rows_before_the_first_position_are_skipped_alone(dv, d, start, n):
    """A chunk that begins before position 0: its other rows are written and read back."""
    H, cu = 2, [0, n[0], n[0] + n[1]]
    pool, table, _ = P.filled(2, H, d, [max(1, a + b) for a, b in zip(start, n)], seed=d)
    pool["ks"].nan_to_num_(0.5)
    pool["vs"].nan_to_num_(0.25)
    k, v = rows(cu[2], H, d, 3), rows(cu[2], H, d, 4)
    c = to_gpu(dv, pool, table)
    dv.dvssq_kv_append(c, k.cuda(), v.cuda(), i32(start), i32(cu))
    assert dv.dvssq_device_error(clear=True) == ERR_INDEX
    ko, vo = torch.full_like(k, 7.0), torch.full_like(v, 9.0)
    kg, vg = ko.cuda(), vo.cuda()
    for b in range(2):                                      # the rows from position 0 on
        cut = min(n[b], max(0, -start[b]))
        at, z = cu[b] + cut, cu[b + 1]
        one = table[b: b + 1]
        P.append(pool, one, k[at:z], v[at:z], [max(0, start[b])], [0, z - at])
        P.read(pool, one, [max(0, start[b])], [0, z - at], ko[at:z], vo[at:z])
    assert torch.equal(c.k.cpu(), pool["k"]) and torch.equal(c.v.cpu(), pool["v"])
    assert torch.equal(c.k_scale.cpu(), pool["ks"]) and torch.equal(c.v_scale.cpu(), pool["vs"])
    dv.dvssq_kv_read(c, i32(start), i32(cu), cu[2], k=kg, v=vg)
    assert dv.dvssq_device_error(clear=True) == ERR_INDEX
    assert torch.equal(kg.cpu(), ko) and torch.equal(vg.cpu(), vo)
