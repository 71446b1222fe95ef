"""Page-cache operators without a GPU: the page bookkeeping against a plain model, the argument
checks of the C ABI, and the 4-bit plan."""

import numpy as np
import pytest
import torch

from cache_ref import E2M1_GRID, E4M3_GRID, nearest, to_e4m3


@pytest.fixture(scope="module", autouse=True)
def pkd():
    from paged_kv_decode_23_gb300 import build
    build.build()


# ------------------------------------------------------------------------------ references
def test_reference_roundings_against_torch():
    x = np.concatenate([np.linspace(-500, 500, 4001), 2.0 ** np.linspace(-14, 9, 999)]).astype(np.float32)
    want = torch.from_numpy(np.clip(x, -448, 448)).to(torch.float8_e4m3fn).double().numpy()
    assert np.array_equal(to_e4m3(x.astype(np.float64)), want)
    assert len(E4M3_GRID) == 127 and E4M3_GRID[-1] == 448
    ties = [0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0]
    assert E2M1_GRID[nearest(np.array(ties), E2M1_GRID)].tolist() == [0, 1, 1, 2, 2, 4, 4]


# ------------------------------------------------------------------------------ bookkeeping
class Model:
    """pkd_pages as plain Python."""

    def __init__(self, n):
        self.uses = [0] * n

    def free_pages(self):
        return [i for i, u in enumerate(self.uses) if u == 0]

    def alloc(self, n):
        got = self.free_pages()[:n]
        for p in got:
            self.uses[p] = 1
        return got


@pytest.mark.parametrize("num_pages", [1, 63, 64, 65, 200])
def test_allocator_follows_a_plain_model(num_pages):
    from paged_kv_decode_23_gb300 import PageAllocator, PkdError
    rng = np.random.default_rng(num_pages)
    a, m, page = PageAllocator(num_pages), Model(num_pages), 8
    tables = []  # (pages, kv_len)
    for step in range(600):
        act = rng.integers(0, 5)
        if act <= 1:
            n = int(rng.integers(0, max(2, num_pages // 6)))
            if n <= len(m.free_pages()):
                got = a.alloc(n)
                assert got.tolist() == m.alloc(n)
                if n:
                    tables.append((got, int(rng.integers((n - 1) * page + 1, n * page + 1))))
            else:
                with pytest.raises(PkdError):
                    a.alloc(n)
        elif act == 2 and tables:
            pages, _ = tables.pop(rng.integers(len(tables)))
            a.free(pages)
            for p in pages:
                m.uses[p] -= 1
        elif act == 3 and tables:
            pages, length = tables[rng.integers(len(tables))]
            kv_len = int(rng.integers(0, length + 1))
            partial = kv_len % page != 0
            if partial and not m.free_pages():
                with pytest.raises(PkdError):
                    a.fork(pages, kv_len, page)
                continue
            child, src, dst = a.fork(pages, kv_len, page)
            full = kv_len // page
            want = list(pages[:full])
            for p in want:
                m.uses[p] += 1
            if partial:
                want += m.alloc(1)
                assert src.tolist() == [pages[full]] and dst.tolist() == [want[-1]]
            else:
                assert len(src) == len(dst) == 0
            assert child.tolist() == want
            if len(child):
                tables.append((child, kv_len))
        elif act == 4 and step % 7 == 0:
            before = {i: u for i, u in enumerate(m.uses) if u}
            src, dst, remap = a.compact()
            assert len(set(dst.tolist())) == len(dst) and not set(src.tolist()) & set(dst.tolist())
            live = len(before)
            assert all(s >= live > d for s, d in zip(src, dst))
            assert {int(remap[i]) for i in before} == set(range(live))
            assert all(remap[s] == d for s, d in zip(src, dst))
            new = [0] * num_pages
            for i, u in before.items():
                new[remap[i]] = u
            m.uses = new
            tables = [(remap[p], n) for p, n in tables]
        assert a.uses().tolist() == m.uses and a.num_free == len(m.free_pages())
    for pages, _ in tables:
        a.free(pages)
    assert a.num_free == num_pages


def test_allocator_refusals_change_nothing():
    from paged_kv_decode_23_gb300 import PageAllocator, PkdError
    a = PageAllocator(10)
    p = a.alloc(4)
    before = a.uses().tolist()
    for bad in ([0, 1, 9], [0, 0], [-1], [10], [2, 2, 2]):
        with pytest.raises(PkdError):
            a.free(bad)
        assert a.uses().tolist() == before and a.num_free == 6
    with pytest.raises(PkdError):
        a.alloc(7)
    with pytest.raises(ValueError):
        a.alloc(11)
    with pytest.raises(PkdError):
        a.fork(p, 65, 16)  # five pages' worth
    with pytest.raises(PkdError):
        a.fork([7], 3, 16)  # not in use
    with pytest.raises(ValueError):
        a.fork(p, -1, 16)
    assert a.uses().tolist() == before
    with pytest.raises(PkdError):
        PageAllocator(-1)
    empty = PageAllocator(0)
    assert empty.num_free == 0 and empty.alloc(0).size == 0 and empty.compact()[0].size == 0
    child, src, dst = a.fork(p, 0, 16)
    assert child.size == src.size == dst.size == 0


# ------------------------------------------------------------------------------ C ABI refusals
def _append_args(**over):
    """A valid pkd_append call's fields (the pointers are never followed on the host)."""
    f = dict(k=4096, v=8192, ks=0, vs=0, pages=8, st=(4096, 256, 128), sst=(0, 0, 0), indptr=64, indices=64,
             n_idx=8, batch=1, dtype=1, hkv=2, d=128, ps=16, k_scale=1.0, v_scale=1.0, q=256, kr=256,
             vr=256, out=256, qst=(512, 128), kst=(256, 128), vst=(256, 128), ost=(512, 128), bi=64, pos=64,
             rp=0, qw=0, kw=0, cs=0, rows=0, status=0, n=1, eps=1e-6, hq=4, in_dtype=1, w32=0, rotary=0,
             inter=0)
    f.update(over)
    from paged_kv_decode_23_gb300 import cache as C
    return C._APPEND.pack(
        f["k"], f["v"], f["ks"], f["vs"], f["pages"], *f["st"], *f["sst"], f["indptr"], f["indices"], f["n_idx"],
        f["batch"], f["dtype"], f["hkv"], f["d"], f["ps"], f["k_scale"], f["v_scale"], 0, f["q"], f["kr"],
        f["vr"], f["out"], *f["qst"], *f["kst"], *f["vst"], *f["ost"], f["bi"], f["pos"], f["rp"], f["qw"],
        f["kw"], f["cs"], f["rows"], f["status"], f["n"], f["eps"], f["hq"], f["in_dtype"], f["w32"],
        f["rotary"], f["inter"], 0)


APPEND_REFUSALS = [
    dict(d=96), dict(ps=12), dict(ps=4), dict(ps=512), dict(hkv=0), dict(pages=0), dict(indptr=0), dict(indices=0),
    dict(k=0), dict(k=4104), dict(st=(4096, 256, 4)), dict(st=(4096, 0, 128)), dict(dtype=0), dict(dtype=7),
    dict(in_dtype=2, dtype=2), dict(k_scale=0.0), dict(v_scale=float("nan")), dict(k_scale=-1.0),
    dict(v_scale=float("inf")), dict(k_scale=1e-30), dict(dtype=3, st=(4096, 128, 64)),
    dict(dtype=3, st=(4096, 128, 64), ks=64, vs=64, sst=(512, 16, 4)),
    dict(dtype=3, st=(4096, 128, 64), ks=65, vs=64, sst=(512, 16, 8)),
    dict(n=-1), dict(hq=0), dict(q=0), dict(kr=0), dict(vr=0), dict(out=0), dict(q=264), dict(qst=(512, 4)),
    dict(bi=0), dict(pos=0), dict(qw=8), dict(eps=-1.0), dict(eps=float("nan")), dict(rotary=8, cs=64),
    dict(rotary=144, cs=64), dict(rotary=64), dict(rotary=64, cs=72), dict(kst=(-256, 128)), dict(batch=-1),
    dict(eps=1e-50), dict(eps=1e300), dict(n=2, ost=(0, 128)), dict(n=3, ost=(504, 128)), dict(ost=(512, 120)),
    dict(n=3, ost=(128, 376)), dict(n=2, ost=(64, 512)),
]


@pytest.mark.parametrize("over", APPEND_REFUSALS, ids=lambda o: ",".join(f"{k}={v}" for k, v in o.items()))
def test_append_refuses(over):
    from paged_kv_decode_23_gb300 import _lib as L
    rc = L.lib().pkd_append(_append_args(**over), None)
    assert rc in (-1, -5) and L.lib().pkd_last_error()


def test_append_and_gather_of_nothing_need_no_device():
    from paged_kv_decode_23_gb300 import _lib as L
    from paged_kv_decode_23_gb300 import cache as C
    assert L.lib().pkd_append(_append_args(n=0), None) == 0
    assert L.lib().pkd_append(None, None) == -1 and L.lib().pkd_gather(None, None) == -1
    pool = (4096, 8192, 0, 0, 8, 4096, 256, 128, 0, 0, 0, 64, 64, 8, 1, 1, 2, 128, 16, 1.0, 1.0, 0)
    assert L.lib().pkd_gather(C._GATHER.pack(*pool, 256, 256, 256, 128, 256, 128, 64, 64, 0, 0, 1, 0), None) == 0
    for bad in ((*pool, 0, 0, 256, 128, 256, 128, 64, 64, 0, 1, 1, 0),      # no output
                (*pool, 264, 0, 256, 128, 256, 128, 64, 64, 0, 1, 1, 0),    # misaligned
                (*pool, 256, 0, 256, 128, 256, 128, 0, 64, 0, 1, 1, 0),     # no batch_indices
                (*pool, 256, 0, 248, 128, 256, 128, 64, 64, 0, 2, 1, 0),    # k's rows overlap
                (*pool, 256, 256, 256, 128, 0, 128, 64, 64, 0, 2, 1, 0),    # v's rows overlap
                (*pool, 256, 0, 256, 128, 256, 128, 64, 64, 0, 1, 0, 0)):   # bf16 cache, fp16 rows
        assert L.lib().pkd_gather(C._GATHER.pack(*bad), None) in (-1, -5)


@pytest.mark.parametrize("src,dst,pages", [([0], [8], 8), ([-1], [1], 8), ([0, 1], [2, 2], 8),
                                           ([0, 1], [1, 2], 8), ([3], [3], 8), ([8], [0], 8)])
def test_copy_pages_refuses(src, dst, pages):
    from paged_kv_decode_23_gb300 import _lib as L
    at = np.array([4096], dtype=np.int64)
    size = np.array([64], dtype=np.int64)
    s, d = np.array(src, dtype=np.int32), np.array(dst, dtype=np.int32)
    rc = L.lib().pkd_copy_pages(at.ctypes.data, size.ctypes.data, size.ctypes.data, 1, pages, s.ctypes.data,
                                d.ctypes.data, len(s), None)
    assert rc == -1 and L.lib().pkd_last_error()


def test_copy_pages_checks_its_pools():
    from paged_kv_decode_23_gb300 import _lib as L
    s, d = np.array([0], dtype=np.int32), np.array([1], dtype=np.int32)

    def call(base, stride, size, n=1, pairs=1):
        b, st, sz = (np.array([x], dtype=np.int64) for x in (base, stride, size))
        return L.lib().pkd_copy_pages(b.ctypes.data, st.ctypes.data, sz.ctypes.data, n, 4, s.ctypes.data,
                                      d.ctypes.data, pairs, None)
    assert call(0, 64, 64) == -1 and call(4096, 32, 64) == -1 and call(4096, 64, -1) == -1
    assert call(4096, 64, 64, n=-1) == -1 and call(4096, 64, 64, pairs=-1) == -1
    assert call(4096, 64, 0) == 0 and call(4096, 64, 64, n=0) == 0 and call(4096, 64, 64, pairs=0) == 0


# ------------------------------------------------------------------------------ Python refusals
def test_python_refuses_host_tensors():
    from paged_kv_decode_23_gb300 import append_paged_kv, copy_pages, gather_paged_kv
    q = torch.zeros(1, 2, 128, dtype=torch.bfloat16)
    i = torch.zeros(1, dtype=torch.int32)
    with pytest.raises(ValueError):
        append_paged_kv(q, q, q, i, i, torch.zeros(2, 2, 16, 2, 128, dtype=torch.bfloat16), i, i)
    with pytest.raises(ValueError):
        append_paged_kv(None, None, None, i, i, None, None, None)
    with pytest.raises(ValueError):
        gather_paged_kv(i, i, torch.zeros(2, 2, 16, 2, 128, dtype=torch.bfloat16), i, i)
    with pytest.raises(ValueError):
        copy_pages([torch.zeros(4, 8)], [0], [1])
    with pytest.raises(ValueError):
        copy_pages([torch.zeros(4, 8)], [0], [1, 2])
    copy_pages([], [], [])


# ------------------------------------------------------------------------------ 4-bit plans
@pytest.mark.parametrize("d", [64, 128, 256])
def test_e2m1_plans_cover_every_token(d):
    from paged_kv_decode_23_gb300 import _lib as L, plan_host
    import workloads as W
    lens = [1, 15, 16, 17, 4000, 0, 129, 777]
    ip, _, lpl, _ = W.page_table(lens, 16)
    plan = plan_host(ip, lpl, 8, 2, d, 16, kv_dtype=L.DTYPE_E2M1)
    assert plan["tile_tokens"] == 128
    got = np.zeros((len(lens), 2), dtype=np.int64)
    for t in plan["tasks"]:
        got[t[0], t[8]] += t[4] - t[3]
    assert np.array_equal(got, np.repeat(np.array(lens)[:, None], 2, axis=1))


def test_e2m1_plan_refusals():
    from paged_kv_decode_23_gb300 import _lib as L, PkdError, plan_host
    ip, lpl = np.array([0, 1], dtype=np.int32), np.array([3], dtype=np.int32)
    with pytest.raises(PkdError):
        plan_host(ip, lpl, 8, 2, 128, 16, kv_dtype=L.DTYPE_E2M1, use_tensor_cores=0)
    with pytest.raises(PkdError):
        plan_host(ip, lpl, 8, 2, 96, 16, kv_dtype=L.DTYPE_E2M1)
    with pytest.raises(PkdError):
        plan_host(ip, lpl, 8, 2, 128, 16, kv_dtype=4)


def test_cos_sin_cache():
    from paged_kv_decode_23_gb300 import make_cos_sin_cache
    t = make_cos_sin_cache(40000, 64, rope_theta=5e5, rope_scale=2.0, device="cpu")
    assert t.shape == (40000, 64) and t.dtype == torch.float32
    for p, i in ((0, 0), (39999, 0), (12345, 7), (39999, 31)):
        angle = p / 2.0 * 5e5 ** (-2 * i / 64)
        assert abs(float(t[p, i]) - np.cos(angle)) <= 2.0 ** -24 and abs(float(t[p, 32 + i]) - np.sin(angle)) <= 2.0 ** -24
    for bad in (0, 8, -16):
        with pytest.raises(ValueError):
            make_cos_sin_cache(10, bad, device="cpu")


def test_packed_structs_have_the_header_s_sizes(tmp_path):
    """The binding packs the argument structs by hand: their sizes and a field's place in each must
    be the C compiler's."""
    import os
    import struct
    import subprocess
    from paged_kv_decode_23_gb300 import cache as C, decode as D
    include = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "include")
    src = tmp_path / "sizes.c"
    src.write_text('#include <stdio.h>\n#include "pkd.h"\nint main(void) { printf("%zu %zu %zu %zu %zu %zu %zu\\n", '
                   "sizeof(pkd_paged_pool), sizeof(pkd_append_args), sizeof(pkd_gather_args), sizeof(pkd_scaled_run), "
                   "offsetof(pkd_append_args, eps), offsetof(pkd_gather_args, out_dtype), offsetof(pkd_scaled_run, q_scale));"
                   " return 0; }\n")
    exe = tmp_path / "sizes"
    subprocess.run(["gcc", "-I", include, str(src), "-o", str(exe)], check=True)
    got = [int(x) for x in subprocess.run([str(exe)], capture_output=True, text=True, check=True).stdout.split()]
    sizes = [struct.Struct("@" + C._POOL).size, C._APPEND.size, C._GATHER.size, D._SCALED_RUN.size]
    assert got[:4] == sizes
    assert got[4:] == [C._APPEND.size - 8 - 24, C._GATHER.size - 8, D._SCALED_RUN.size - 16]


@pytest.mark.parametrize("kind", ["list", "numpy", "tensor"])
@pytest.mark.parametrize("ids", [[2 ** 32], [2 ** 32 + 1, 0], [-2 ** 32], [0.5], [1.0], [2 ** 31]])
def test_page_ids_of_more_than_32_bits_are_refused(kind, ids):
    """Not taken modulo 2^32, nor cut to whole numbers: page 0 would lose a use, or be copied."""
    from paged_kv_decode_23_gb300 import PageAllocator, copy_pages
    x = {"list": lambda: ids, "numpy": lambda: np.array(ids), "tensor": lambda: torch.tensor(ids)}[kind]()
    a = PageAllocator(4)
    a.alloc(2)
    with pytest.raises(ValueError):
        a.free(x)
    with pytest.raises(ValueError):
        a.fork(x, 3, 16)
    assert a.uses().tolist() == [1, 1, 0, 0]
    for pair in ((x, list(range(2, 2 + len(ids)))), (list(range(2, 2 + len(ids))), x)):
        with pytest.raises(ValueError, match="32-bit"):
            copy_pages([torch.zeros(4, 8)], *pair)
    a.free(np.array([1], dtype=np.int64))
    a.free(torch.tensor([0], dtype=torch.int16))
    a.free([])
    assert a.num_free == 4


# ------------------------------------------------------------------------------ rows that overlap
def _starts(at, st, n, heads):
    return (at // 2 + st[0] * np.arange(n)[:, None] + st[1] * np.arange(heads)).ravel()


def _meet(a, b, d):
    return bool((np.abs(a[:, None] - b) < d).any())


@pytest.mark.parametrize("over", APPEND_REFUSALS, ids=lambda o: ",".join(f"{k}={v}" for k, v in o.items()))
def test_append_refuses_where_rows_lie_apart(over):
    """As above, with k and v away from q: it is the argument that is refused."""
    from paged_kv_decode_23_gb300 import _lib as L
    args = _append_args(**{**dict(kr=1 << 20, vr=2 << 20, out=256), **over})
    assert L.lib().pkd_append(args, None) in (-1, -5)
    assert b"q_out overlaps" not in L.lib().pkd_last_error()


def test_append_rows_that_overlap():
    """q_out against q, k and v in layouts of many kinds, against all pairs of rows.  (Without batch
    indices: no call gets as far as a launch.)"""
    from paged_kv_decode_23_gb300 import _lib as L
    rng = np.random.default_rng(2)
    d, base, seen = 64, 1 << 22, [0, 0]
    for step in range(3000):
        n, hq, hkv = (int(x) for x in rng.integers(1, 5, 3))
        kind = rng.integers(4)
        if kind == 0:  # one projection's output
            row = (hq + 2 * hkv) * d
            st = {x: (row, d) for x in "qkvo"}
            at = dict(q=0, k=hq * d, v=(hq + hkv) * d, o=0)
        elif kind == 1:  # q, k and v of a kv head together
            hq = hkv
            st = {x: (3 * hkv * d, 3 * d) for x in "qkvo"}
            at = dict(q=0, k=d, v=2 * d, o=0)
        elif kind == 2:  # heads first
            st = {x: (d, n * d) for x in "qkvo"}
            at = dict(q=0, k=hq * n * d, v=(hq + hkv) * n * d, o=0)
        else:
            st = {x: (int(rng.integers(hq + hkv, 12)) * d, d) for x in "qkvo"}
            at = {x: int(rng.integers(0, 40)) * d for x in "qkvo"}
        if rng.random() < 0.5:
            at["o"] += int(rng.integers(-40, 40)) * d // 2 // 8 * 8
        if rng.random() < 0.3:
            at["o"] += 100 * d
        if rng.random() < 0.2:
            st["o"] = (hq * d, d)
        at = {x: base + 2 * v for x, v in at.items()}
        out = _starts(at["o"], st["o"], n, hq)
        own = [_meet(out[:i], out[i:i + 1], d) for i in range(1, len(out))]
        if any(own):
            continue
        same = at["o"] == at["q"] and (n == 1 or st["o"][0] == st["q"][0]) and (hq == 1 or st["o"][1] == st["q"][1])
        want = (not same and _meet(out, _starts(at["q"], st["q"], n, hq), d)) or any(
            _meet(out, _starts(at[x], st[x], n, hkv), d) for x in "kv")
        args = _append_args(n=n, hq=hq, hkv=hkv, d=d, st=(1 << 14, 1 << 10, d), q=at["q"], kr=at["k"], vr=at["v"],
                            out=at["o"], qst=st["q"], kst=st["k"], vst=st["v"], ost=st["o"], bi=0)
        assert L.lib().pkd_append(args, None) == -1
        msg = L.lib().pkd_last_error()
        got = b"q_out overlaps" in msg
        assert got or b"null batch_indices" in msg, msg
        seen[want] += 1
        if want:
            assert got
        elif got:  # refused unread: tokens at different distances in the memory of another's
            assert n > 1 and len({st["o"][0], st["q"][0], st["k"][0], st["v"][0]}) > 1
    assert min(seen) > 300


def test_gather_outputs_that_overlap():
    from paged_kv_decode_23_gb300 import _lib as L
    from paged_kv_decode_23_gb300 import cache as C
    pool = (4096, 8192, 0, 0, 8, 4096, 256, 128, 0, 0, 0, 64, 64, 8, 1, 1, 2, 128, 16, 1.0, 1.0, 0)

    def call(k, v, kst, vst, n=3):  # (no batch indices: no call gets as far as a launch)
        assert L.lib().pkd_gather(C._GATHER.pack(*pool, k, v, *kst, *vst, 0, 64, 0, n, 1, 0), None) == -1
        return L.lib().pkd_last_error()
    for k, v, kst, vst in ((4096, 4096, (256, 128), (256, 128)), (4096, 4352, (256, 128), (256, 128)),
                           (4096, 4096 + 2 * 384, (512, 128), (512, 128)), (4096, 4112, (1024, 128), (1024, 128)),
                           (8192, 4096 + 2 * 300 // 8 * 8 * 8, (512, 128), (512, 256))):
        assert b"overlaps v_out" in call(k, v, kst, vst)
    for k, v, kst, vst in ((4096, 4096 + 2 * 768, (256, 128), (256, 128)), (4096, 4096 + 512, (512, 128), (512, 128)),
                           (4096, 4096 + 256, (512, 256), (512, 256)), (1 << 20, 4096, (256, 128), (256, 128))):
        assert b"null batch_indices" in call(k, v, kst, vst)


def test_allocator_arguments_of_more_bits_than_the_library_s():
    """Cut to the library's types they would be other, valid numbers: fork would write more page ids than
    its output holds."""
    from paged_kv_decode_23_gb300 import PageAllocator, PkdError
    a = PageAllocator(8)
    p = a.alloc(8)
    for kv_len, page_size in ((2 ** 64 + 5, 16), (2 ** 63, 16), (5, 2 ** 32 + 1), (5, 2 ** 31), (100, 2 ** 32 + 16)):
        with pytest.raises(ValueError):
            a.fork(p, kv_len, page_size)
    with pytest.raises(PkdError):
        a.fork(p, 2 ** 63 - 1, 2 ** 31 - 1)
    for n in (2 ** 31, 2 ** 64 + 4):
        with pytest.raises(ValueError):
            PageAllocator(n)
    assert a.uses().tolist() == [1] * 8


@pytest.mark.parametrize("over", [
    dict(v=4096), dict(st=(4096, 128, 128)), dict(st=(2048, 256, 128)), dict(st=(4096, 256, 64)), dict(st=(128, 2048, 512)),
    dict(dtype=3, st=(4096, 128, 32), ks=64, vs=4096, sst=(512, 16, 8)),
    dict(dtype=3, st=(4096, 128, 64), ks=64, vs=4096, sst=(512, 8, 8)),
    dict(dtype=3, st=(4096, 128, 64), ks=64, vs=64, sst=(512, 16, 8)),
], ids=str)
def test_append_into_a_pool_that_overlaps_itself(over):
    from paged_kv_decode_23_gb300 import _lib as L
    # (without batch indices: no call gets as far as a launch)
    assert L.lib().pkd_append(_append_args(**{**dict(kr=1 << 20, vr=2 << 20, bi=0), **over}), None) == -1
    assert b"overlap" in L.lib().pkd_last_error()


@pytest.mark.parametrize("over", [
    dict(), dict(st=(4096, 128, 2048)), dict(st=(256, 4096, 128)), dict(st=(128, 2048, 1024)), dict(hkv=1, st=(4096, 256, 8)),
    dict(pages=1, st=(8, 256, 128)), dict(dtype=2, st=(4096, 256, 128)), dict(dtype=3, st=(2048, 128, 64), ks=64, vs=4096, sst=(256, 16, 8)),
], ids=str)
def test_append_into_pools_of_any_axis_order(over):
    from paged_kv_decode_23_gb300 import _lib as L
    assert L.lib().pkd_append(_append_args(**{**dict(kr=1 << 20, vr=2 << 20, bi=0), **over}), None) == -1
    assert b"null batch_indices" in L.lib().pkd_last_error()
