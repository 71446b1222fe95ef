"""Windows with sinks, key weights and eviction without a GPU: the planner's partition, the refusals
and the C ABI's checks."""
import numpy as np
import pytest
import torch  # noqa: F401


@pytest.fixture(scope="module", autouse=True)
def pkd():
    from paged_kv_decode_23_gb300 import build
    build.build()


def _table(lens, page):
    lens = np.asarray(lens, dtype=np.int64)
    pages = -(-lens // page)
    indptr = np.zeros(len(lens) + 1, dtype=np.int32)
    np.cumsum(pages, out=indptr[1:])
    return indptr, np.where(lens > 0, lens - (pages - 1) * page, 0).astype(np.int32)


def _check(lens, page, plan, indptr, hkv, window, sinks, q_len, fixed=0):
    tasks, merges = plan["tasks"], plan["merges"]
    units, slots = {}, []
    for t in tasks:
        units.setdefault((int(t[0]), int(t[8]), int(t[9])), []).append(t)
    gsl = 1 + int(tasks[:, 9].max(initial=0))
    assert len(units) == len(lens) * q_len * hkv * gsl
    for (row, kvh, gs), ts in units.items():
        n = max(0, int(lens[row // q_len]) - (q_len - 1 - row % q_len))
        want = [t for t in range(n) if window < 0 or t >= n - 1 - window or t < sinks]
        got = []
        for t in sorted(ts, key=lambda t: int(t[5])):
            c0, b, e, s0, s1 = (int(t[i]) for i in (2, 3, 4, 12, 13))
            assert int(t[1]) == indptr[row // q_len]
            assert n == 0 or int(t[7]) == n - 1
            assert c0 % page == 0 and c0 <= b and s0 % page == 0 and 0 <= s0 <= s1
            assert s1 == 0 or (s1 > s0 and s1 == min(sinks, s1) and s1 < b < e)  # never sinks alone
            if fixed:
                assert c0 % fixed == 0 and e - c0 <= fixed and s0 % fixed == 0 and s1 - s0 < fixed
            got += list(range(s0, s1)) + list(range(b, e))
            assert n == 0 or e > b
        assert got == want, (row, n, ts)
        if len(ts) == 1:
            assert ts[0][5] == -1 and ts[0][6] == -1
        else:
            m = merges[int(ts[0][6])]
            assert int(m[0]) == row and int(m[2]) == len(ts) and int(m[3]) == kvh * gsl + gs
            mine = sorted(int(t[5]) for t in ts)
            assert mine == list(range(int(m[1]), int(m[1]) + len(ts)))
            slots += mine
    assert sorted(slots) == list(range(plan["num_slots"]))
    long = tasks[:, 4] - tasks[:, 3] + tasks[:, 13] - tasks[:, 12]
    assert np.all(np.diff(long) <= 0)


@pytest.mark.parametrize("seed", range(60))
def test_plans_with_sinks_partition_the_attended_tokens(seed):
    from paged_kv_decode_23_gb300 import plan_host
    rng = np.random.default_rng(seed)
    page = int(rng.choice([8, 16, 64, 256]))
    batch = int(rng.choice([1, 2, 5, 40, 200]))
    top = int(rng.choice([20, 700, 5000]))
    lens = rng.integers(0, top + 1, batch)
    window = int(rng.integers(0, top))
    sinks = int(rng.choice([1, 4, 16, 17, 100, 300, 1000, 2 ** 31 - 1]))
    q_len = int(rng.choice([1, 1, 3]))
    hkv, group = int(rng.choice([1, 2, 8])), int(rng.choice([1, 4, 12]))
    mode = int(rng.integers(0, 3))
    kw = {} if mode == 0 else dict(fixed_split_size=int(rng.integers(1, 5))) if mode == 1 else dict(disable_split_kv=True)
    d = int(rng.choice([64, 128, 256]))
    indptr, last = _table(lens, page)
    plan = plan_host(indptr, last, hkv * group, hkv, d, page, window_left=window, num_sink_tokens=sinks,
                     q_len_per_req=q_len, kv_dtype=int(rng.choice([0, 1, 3])), **kw)
    _check(lens, page, plan, indptr, hkv, window, sinks, q_len, kw.get("fixed_split_size", 0) * page)


@pytest.mark.parametrize("window,sinks", [(-1, 7), (5000, 4), (99, 400)])
def test_sinks_without_a_gap_change_nothing(window, sinks):
    from paged_kv_decode_23_gb300 import plan_host
    lens = [400, 1, 0, 77, 300]
    indptr, last = _table(lens, 16)
    a = plan_host(indptr, last, 32, 8, 128, 16, window_left=window, num_sink_tokens=sinks)
    b = plan_host(indptr, last, 32, 8, 128, 16, window_left=-1)
    assert np.array_equal(a["tasks"][:, :12], b["tasks"]) and np.array_equal(a["merges"], b["merges"])
    assert (a["tasks"][:, 12:] == 0).all()


def test_a_fixed_split_with_sinks_does_not_depend_on_the_batch():
    from paged_kv_decode_23_gb300 import plan_host
    lens = [5000, 300, 2111]
    kw = dict(window_left=1000, num_sink_tokens=150, fixed_split_size=4)

    def parts(lens, i):
        indptr, last = _table(lens, 16)
        t = plan_host(indptr, last, 4, 1, 128, 16, **kw)["tasks"]
        t = t[t[:, 0] == i]
        return sorted(map(tuple, t[:, [2, 3, 4, 12, 13]].tolist()))

    for i, n in enumerate(lens):
        assert parts(lens, i) == parts([n], 0)


def test_a_work_list_of_a_capacity_holds_sinks():
    from paged_kv_decode_23_gb300 import plan_host
    lens = [9000, 20, 4000]
    indptr, last = _table(lens, 16)
    plan = plan_host(indptr, last, 8, 2, 128, 16, window_left=3000, num_sink_tokens=700, work_capacity=5)
    assert len(plan["tasks"]) <= 5 * 2
    _check(lens, 16, plan, indptr, 2, 3000, 700, 1)


@pytest.mark.parametrize("bad", [-1, -2 ** 31, 2 ** 31, 2 ** 40])
def test_numbers_of_sinks_that_are_refused(bad):
    from paged_kv_decode_23_gb300 import PkdError, plan_host, workspace_bytes
    indptr, last = _table([100], 16)
    for call in (plan_host, workspace_bytes):
        with pytest.raises((PkdError, ValueError)):
            call(indptr, last, 8, 2, 128, 16, window_left=10, num_sink_tokens=bad)


def test_null_arguments_are_refused():
    from paged_kv_decode_23_gb300 import _lib as L
    assert L.lib().pkd_plan_with(None, None, None) == -1
    assert L.lib().pkd_plan_tasks(None, 152, 0, None, 0, None, 0, None, None, None) == -1
    assert L.lib().pkd_plan_workspace_bytes(None, 152, None, None) == -1


def test_workspace_bytes_of_a_plan_with_sinks_are_those_of_what_it_attends():
    from paged_kv_decode_23_gb300 import workspace_bytes
    indptr, last = _table([50000, 300], 16)
    whole = workspace_bytes(indptr, last, 32, 8, 128, 16)
    part = workspace_bytes(indptr, last, 32, 8, 128, 16, window_left=1000, num_sink_tokens=16)
    assert 0 < part[0] <= whole[0] and 0 < part[1] <= whole[1]


def test_key_weight_plans_that_are_refused_and_what_they_take():
    from paged_kv_decode_23_gb300 import PkdError, graph_workspace_bytes, workspace_bytes
    lens = [5000, 0, 77]
    indptr, last = _table(lens, 16)
    plain = workspace_bytes(indptr, last, 32, 8, 128, 16)
    with_keys = workspace_bytes(indptr, last, 32, 8, 128, 16, key_weights=True)
    scores = 32 * sum(-(-n // 16) * 16 for n in lens) * 4
    assert scores <= with_keys[0] - plain[0] <= scores + 2048 and with_keys[1] > plain[1]
    bounded = workspace_bytes(indptr, last, 32, 8, 128, 16, key_weights=True, window_left=255, num_sink_tokens=4)
    assert bounded[0] < plain[0] + 32 * 4 * (5000 // 4)
    with pytest.raises(PkdError, match="UNSUPPORTED"):
        workspace_bytes(indptr, last, 32, 8, 128, 16, key_weights=True, use_tensor_cores=0)
    a, b = graph_workspace_bytes(400, 32, 8, 128), graph_workspace_bytes(400, 32, 8, 128, key_weights_pages=500, page_size=16, max_batch=8)
    assert b[0] - a[0] >= 500 * 16 * 32 * 4 and b[1] > a[1]
    for bad in (dict(key_weights_pages=-1, page_size=16, max_batch=8), dict(key_weights_pages=5, page_size=0, max_batch=8)):
        with pytest.raises(PkdError):
            graph_workspace_bytes(400, 32, 8, 128, **bad)


@pytest.mark.parametrize("seed", range(12))
def test_the_graph_workspace_covers_every_plan(seed):
    """What plans of a capacity need stays inside the two bounds together."""
    from paged_kv_decode_23_gb300 import graph_workspace_bytes, workspace_bytes
    rng = np.random.default_rng(seed)
    page, q_len, group = int(rng.choice([8, 16, 256])), int(rng.choice([1, 3])), int(rng.choice([1, 4, 12]))
    batch = int(rng.integers(1, 9))
    lens = rng.integers(0, 3000, batch)
    indptr, last = _table(lens, page)
    items = batch * q_len + 304
    kw = dict(window_left=int(rng.integers(0, 2000)), num_sink_tokens=int(rng.choice([0, 3, 100])), q_len_per_req=q_len)
    need = workspace_bytes(indptr, last, 2 * group, 2, 128, page, key_weights=True, **kw)
    base = workspace_bytes(indptr, last, 2 * group, 2, 128, page, **kw)
    have = graph_workspace_bytes(items, 2 * group, 2, 128, key_weights_pages=int(indptr[-1]), page_size=page, max_batch=batch,
                                 q_len_per_req=q_len)
    floor = graph_workspace_bytes(items, 2 * group, 2, 128)
    assert have[0] - floor[0] >= need[0] - base[0] and have[1] - floor[1] >= need[1] - base[1]


def _evict_args(**over):
    """pkd_evict_args with made-up device addresses: for calls that fail before any launch."""
    from paged_kv_decode_23_gb300 import cache
    f = dict(k=4096, v=8192, ks=0, vs=0, pages=10, s0=4096, s1=256, s2=128, f0=0, f1=0, f2=0, ip=64, ix=64, nidx=9, batch=2,
             dtype=1, hkv=2, d=128, ps=16, kscale=1.0, vscale=1.0, r=0, w=256, w0=32, w1=16, w2=1, lens=64, kept=0, moves=64,
             status=0, budget=64, sinks=4, recent=8, r2=0)
    f.update(over)
    return cache._EVICT.pack(*f.values())


@pytest.mark.parametrize("over,code", [
    (dict(budget=0), -1), (dict(budget=-3), -1), (dict(budget=2 ** 30 + 1), -1), (dict(budget=2 ** 31 - 1), -1), (dict(sinks=-1), -1), (dict(recent=-1), -1), (dict(sinks=60), -1),
    (dict(recent=2 ** 31 - 1, sinks=2 ** 31 - 1), -1), (dict(w=0), -1), (dict(w=258), -1), (dict(w2=0), -1), (dict(w0=15), -1),
    (dict(w1=-16), -1), (dict(w0=2 ** 62), -1), (dict(lens=0), -1), (dict(moves=0), -1), (dict(moves=68), -1), (dict(ip=0), -1),
    (dict(ix=0), -1), (dict(k=0), -1), (dict(v=4096), -1), (dict(k=4100), -1), (dict(s1=100), -1), (dict(s0=128), -1),
    (dict(dtype=3), -1), (dict(dtype=7), -5), (dict(d=96), -5), (dict(ps=12), -5), (dict(hkv=0), -1), (dict(batch=-1), -1),
    (dict(pages=0), -1), (dict(batch=2 ** 20, hkv=2 ** 12), -1),
])
def test_evictions_that_are_refused(over, code):
    from paged_kv_decode_23_gb300 import _lib as L
    assert L.lib().pkd_evict(_evict_args(**over), None) == code, L.lib().pkd_last_error()


def test_an_eviction_of_nothing_needs_no_gpu():
    from paged_kv_decode_23_gb300 import _lib as L
    assert L.lib().pkd_evict(None, None) == -1
    assert L.lib().pkd_evict(_evict_args(batch=0), None) == 0


@pytest.mark.parametrize("at,name", [(4, "sm_scale"), (5, "logits_soft_cap"), (6, "rope_scale"), (7, "rope_theta")])
def test_numbers_past_32_bits_reach_the_plan_as_infinite(at, name):
    """(which refuses them, as one call of pkd_plan with 32-bit arguments did)"""
    import struct
    from paged_kv_decode_23_gb300 import decode
    fields = [0] * 4 + [0.5, 1.0, 2.0, 1e4] + [1] * 16
    fields[at] = 1e300
    got = struct.unpack("@3Pq4f16i", decode._plan_args(*fields))
    assert got[at] == float("inf") and got[:at] == tuple(fields[:at]) and got[at + 1:] == tuple(fields[at + 1:])
    with pytest.raises(ValueError, match="32 bits"):
        decode._plan_args(*fields[:8], 2 ** 31, *fields[9:])
