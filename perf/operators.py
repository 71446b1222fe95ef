"""Cases of the operators around a paged KV cache: what is measured, in plain torch and through
this package's entry points.

  append  rms-norm and rotate the new queries and keys, write K and V into their page slots
  decode  decode attention over a cache held in 4 bits (e2m1 values, an e4m3 scale per 16)
  gather  read listed tokens of a cache back as 16-bit rows
  copy    copy pages of every layer's pool (forked sequences, compaction)
"""
import math

import numpy as np
import torch

own = False

DT = {"bf16": torch.bfloat16, "f16": torch.float16, "e4m3": torch.float8_e4m3fn}
E2M1 = (0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0)
EPS = 1e-6


# ------------------------------------------------------------------------------------ cases
def listed():
    return [
        # the newest token of one chat, one layer: nothing but latency
        dict(name="append one token", op="append", dtype="bf16", kv="bf16", layout="NHD", hq=32,
             hkv=8, d=128, page=16, batch=1, new=1, ctx=500, pad=0, norm=True, rotary=128,
             interleaved=False),
        # a decode step of 61 sequences in a batch padded to 64, into a 4-bit cache
        dict(name="append step 4-bit", op="append", dtype="bf16", kv="e2m1", layout="HND", hq=32,
             hkv=8, d=128, page=16, batch=61, new=1, ctx=1000, pad=3, norm=True, rotary=128,
             interleaved=False),
        # seven prompts of very different lengths enter an empty 16-bit cache
        dict(name="append prompts", op="append", dtype="f16", kv="f16", layout="NHD", hq=64,
             hkv=8, d=128, page=16, batch=7, new=1170, ctx=0, pad=0, norm=True, rotary=128,
             interleaved=False),
        # later chunks of long prompts: 8-bit cache, wide heads, a quarter of each rotated
        dict(name="append chunk 8-bit", op="append", dtype="bf16", kv="e4m3", layout="NHD", hq=16,
             hkv=2, d=256, page=32, batch=5, new=819, ctx=1500, pad=0, norm=True, rotary=64,
             interleaved=True),
        # one sequence decodes its next token
        dict(name="decode one", op="decode", dtype="bf16", layout="HND", hq=32, hkv=8, d=128,
             page=16, batch=1, lo=777, hi=777, cap=0.0, window=-1),
        # the framework's headline batch, its cache in 4 bits
        dict(name="decode batch", op="decode", dtype="bf16", layout="NHD", hq=32, hkv=8, d=128,
             page=16, batch=64, lo=512, hi=4096, cap=0.0, window=-1),
        # few very long sequences: each is split over the whole GPU
        dict(name="decode long", op="decode", dtype="f16", layout="HND", hq=32, hkv=8, d=128,
             page=64, batch=4, lo=131072, hi=131072, cap=0.0, window=-1),
        # wide heads, soft cap and sliding window, lengths from one token on
        dict(name="decode window", op="decode", dtype="bf16", layout="NHD", hq=16, hkv=2, d=256,
             page=32, batch=128, lo=1, hi=8192, cap=30.0, window=4096),
        # the short cached prefixes of three sequences, before their next chunk's prefill
        dict(name="gather short", op="gather", dtype="bf16", kv="e4m3", layout="NHD", hkv=2, d=256,
             page=32, batch=3, tokens=901, pad=0),
        # long cached prefixes out of a 4-bit cache
        dict(name="gather prefixes", op="gather", dtype="bf16", kv="e2m1", layout="HND", hkv=8,
             d=128, page=16, batch=16, tokens=65536, pad=0),
        # four sequences fork: their partly filled last pages are copied in every layer
        dict(name="copy fork", op="copy", kv="e2m1", layout="HND", hkv=8, d=128, page=16, layers=8,
             pool=200, pairs=4),
        # a fragmented cache is compacted
        dict(name="copy compact", op="copy", kv="bf16", layout="NHD", hkv=8, d=128, page=16,
             layers=6, pool=4500, pairs=2000),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["append", "append", "decode", "decode", "gather", "copy"])
    d = rng.choice([64, 128, 128, 256])
    hkv = rng.choice([1, 2, 3, 4, 8])
    page = rng.choice([8, 16, 32, 64])
    layout = rng.choice(["NHD", "HND"])
    dtype = rng.choice(["bf16", "f16"])
    kv = rng.choice([dtype, "e4m3", "e2m1"])
    if op == "append":
        group = rng.choice([1, 3, 4, 8])
        t = _log(rng, 1, 8000 * 8 * 128 // (8 * max(128, hkv * d // 4 * group // 2)) + 1)
        t = min(t, 8000)
        step = t <= 256 and rng.random() < 0.5
        batch = t if step else min(t, rng.randint(1, 9))
        return dict(op=op, dtype=dtype, kv=kv, layout=layout, hq=hkv * group, hkv=hkv, d=d,
                    page=page, batch=batch, new=max(1, t // batch),
                    ctx=_log(rng, 1, 60000 // batch + 1), pad=rng.choice([0, 0, 1, 5]),
                    norm=rng.random() < 0.75, rotary=rng.choice([d, d, d // 2, 16, 0]),
                    interleaved=rng.random() < 0.3)
    if op == "decode":
        batch = _log(rng, 1, 128)
        hi = _log(rng, 1, max(2, min(131072, 500000 * 8 * 128 // (batch * hkv * d))))
        return dict(op=op, dtype=dtype, layout=layout, hq=hkv * rng.choice([1, 4, 6, 8, 12]),
                    hkv=hkv, d=d, page=page, batch=batch, lo=rng.randint(1, hi), hi=hi,
                    cap=rng.choice([0.0, 0.0, 30.0]),
                    window=rng.choice([-1, -1, rng.randint(0, hi)]))
    if op == "gather":
        t = _log(rng, 1, 60000 * 8 * 128 // (max(8, hkv) * max(128, d)))
        return dict(op=op, dtype=dtype, kv=kv, layout=layout, hkv=hkv, d=d, page=page,
                    batch=min(t, rng.randint(1, 20)), tokens=t, pad=rng.choice([0, 0, 7]))
    pool = _log(rng, 8, 3000)
    return dict(op=op, kv=kv, layout=layout, hkv=hkv, d=d, page=page, layers=rng.randint(1, 6),
                pool=pool, pairs=rng.randint(1, pool // 2))


def _pool_bytes(c):  # of one token and kv head, K alone
    return {"e2m1": c["d"] // 2 + c["d"] // 16, "e4m3": c["d"]}.get(c["kv"], 2 * c["d"])


def _attended(c):
    n = _decode_lens(c)
    return int((np.minimum(n, c["window"] + 1) if c["window"] >= 0 else n).sum())


def work(case):
    c = case
    if c["op"] == "append":
        t = c["batch"] * c["new"]
        rows = c["hq"] + 2 * c["hkv"]
        return {"bytes": t * (rows * c["d"] * 2 + c["hq"] * c["d"] * 2 + 2 * c["hkv"] * _pool_bytes(c)
                              + 4 * c["rotary"] + 12),
                "flops": t * (c["hq"] + c["hkv"]) * c["d"] * (4 + 3)}
    if c["op"] == "decode":
        a = _attended(c)
        kv = a * c["hkv"] * 2 * (c["d"] // 2 + c["d"] // 16)
        return {"bytes": kv + c["batch"] * c["hq"] * (4 * c["d"] + 4) + 4 * (a // c["page"] + c["batch"]),
                "flops": 4 * a * c["hq"] * c["d"]}
    if c["op"] == "gather":
        return {"bytes": c["tokens"] * (2 * c["hkv"] * (_pool_bytes(c) + 2 * c["d"]) + 12), "flops": 0}
    return {"bytes": 2 * c["layers"] * c["pairs"] * 2 * c["page"] * c["hkv"] * _pool_bytes(c), "flops": 0}


# ------------------------------------------------------------------------------------ inputs
def _gen(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    return g


def _randn(g, *shape):
    return torch.randn(shape, generator=g, device="cuda", dtype=torch.float32)


def _shape(c, pages, width):
    if c["layout"] == "NHD":
        return (pages, 2, c["page"], c["hkv"], width)
    return (pages, 2, c["hkv"], c["page"], width)


def _make_pool(c, g, pages):
    """A pool of normal values: (values, None), or (packed e2m1 codes, e4m3 scales)."""
    if c.get("kv", "e2m1") != "e2m1":
        x = torch.empty(_shape(c, pages, c["d"]), dtype=DT[c["kv"]], device="cuda")
        for p in range(0, pages, 1024):
            x[p:p + 1024] = _randn(g, *x[p:p + 1024].shape).to(x.dtype)
        return x, None
    data = torch.empty(_shape(c, pages, c["d"] // 2), dtype=torch.uint8, device="cuda")
    scales = torch.empty(_shape(c, pages, c["d"] // 16), dtype=DT["e4m3"], device="cuda")
    mids = torch.tensor([0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0], device="cuda")
    for p in range(0, pages, 1024):
        x = _randn(g, *scales[p:p + 1024].shape, 16)
        s = (x.abs().amax(-1) / 6.0).to(DT["e4m3"])
        codes = torch.bucketize(x.abs() / s.float().unsqueeze(-1), mids, out_int32=True)
        codes = (codes + 8 * (x < 0)).to(torch.uint8).view(*data[p:p + 1024].shape, 2)
        data[p:p + 1024] = codes[..., 0] | (codes[..., 1] << 4)
        scales[p:p + 1024] = s
    return data, scales


def _page_table(rng, lens, page, pool):
    """CSR page table: each sequence's pages are drawn without order from a pool of `pool` pages."""
    pages = -(-lens // page)
    indptr = np.zeros(len(lens) + 1, dtype=np.int32)
    np.cumsum(pages, out=indptr[1:])
    indices = rng.permutation(pool)[:int(indptr[-1])].astype(np.int32)
    last = np.where(lens > 0, lens - (pages - 1) * page, 0).astype(np.int32)
    return indptr, indices, last


def _decode_lens(c):
    return np.rint(np.linspace(c["lo"], c["hi"], c["batch"])).astype(np.int64)


def _split(rng, total, parts):
    """`total` cut into `parts` numbers of at least one, of very different sizes."""
    w = rng.exponential(size=parts) + 0.05
    n = 1 + np.floor((total - parts) * w / w.sum()).astype(np.int64)
    n[0] += total - n.sum()
    return n


def _cos_sin(positions, rotary, theta=1e4):
    rate = theta ** (-torch.arange(0, rotary, 2, dtype=torch.float64, device="cuda") / rotary)
    a = torch.arange(positions, dtype=torch.float64, device="cuda").unsqueeze(1) * rate
    return torch.cat([a.cos(), a.sin()], dim=1).float()


def _dev(a):
    return torch.from_numpy(np.ascontiguousarray(a)).cuda()


def _tokens(s, batch, pos, pad):
    """Token rows as the batch lists them, `pad` rows behind the last one."""
    s["batch_indices"] = _dev(np.concatenate([batch, np.full(pad, -1)]).astype(np.int32))
    s["positions"] = _dev(np.concatenate([pos, np.zeros(pad)]).astype(np.int32))
    s["tokens"] = len(batch)


def _inputs(c, seed):
    rng, g = np.random.default_rng(seed), _gen(seed)
    s = {"case": c}
    if c["op"] == "append":
        t, b = c["batch"] * c["new"], c["batch"]
        new = _split(rng, t, b)
        ctx = rng.integers(0, 2 * c["ctx"], b, endpoint=True)
        pool = (2 * c["ctx"] * b + t) // c["page"] + b + 1
        indptr, indices, _ = _page_table(rng, ctx + new, c["page"], pool)
        _tokens(s, np.repeat(np.arange(b), new),
                np.concatenate([np.arange(x, x + n) for x, n in zip(ctx, new)]), c["pad"])
        rows, dt = t + c["pad"], DT[c["dtype"]]
        # one projection's output, as a model hands it over: q, k and v are views of it
        qkv = _randn(g, rows, c["hq"] + 2 * c["hkv"], c["d"]).to(dt)
        s["q"], s["k"], s["v"] = qkv.split([c["hq"], c["hkv"], c["hkv"]], dim=1)
        s["q_out"] = torch.zeros(rows, c["hq"], c["d"], dtype=dt, device="cuda")
        if c["norm"]:
            s["q_weight"], s["k_weight"] = (1 + 0.2 * _randn(g, 2, c["d"])).to(dt).unbind(0)
        if c["rotary"]:
            s["cos_sin"] = _cos_sin(int((ctx + new).max()) + 1, c["rotary"])
    elif c["op"] == "decode":
        lens = rng.permutation(_decode_lens(c))
        pool = int(1.1 * (-(-lens // c["page"])).sum()) + 1
        indptr, indices, last = _page_table(rng, lens, c["page"], pool)
        s["q"] = _randn(g, c["batch"], c["hq"], c["d"]).to(DT[c["dtype"]])
        s["lens"], s["last"] = lens, torch.from_numpy(last)
        s["host_indptr"] = torch.from_numpy(indptr)
        width = int(np.diff(indptr).max())  # the same pages as a padded table, for the plain form
        table = np.zeros((c["batch"], width), dtype=np.int64)
        for i in range(c["batch"]):
            table[i, :indptr[i + 1] - indptr[i]] = indices[indptr[i]:indptr[i + 1]]
        s["table"], s["dev_lens"] = _dev(table), _dev(lens)
    elif c["op"] == "gather":
        n = _split(rng, c["tokens"], c["batch"])
        pool = int(1.3 * c["tokens"]) // c["page"] + c["batch"] + 1
        indptr, indices, _ = _page_table(rng, n, c["page"], pool)
        _tokens(s, np.repeat(np.arange(c["batch"]), n), np.concatenate([np.arange(x) for x in n]), c["pad"])
        shape = (c["tokens"] + c["pad"], c["hkv"], c["d"])
        s["k_out"], s["v_out"] = (torch.zeros(shape, dtype=DT[c["dtype"]], device="cuda") for _ in range(2))
    else:
        order = rng.permutation(c["pool"]).astype(np.int32)
        s["src"], s["dst"] = (torch.from_numpy(x.copy()) for x in (order[:c["pairs"]], order[-c["pairs"]:]))
        s["dev_src"], s["dev_dst"] = s["src"].cuda().long(), s["dst"].cuda().long()
        pools = [x for _ in range(c["layers"]) for x in _make_pool(c, g, c["pool"])]
        s["pools"] = [x for x in pools if x is not None]
        return s
    if c.get("kv") == "e4m3" or c["op"] == "decode" or c.get("kv") == "e2m1":
        s["k_scale"], s["v_scale"] = 0.75, 1.25
    s["indptr"], s["indices"] = _dev(indptr), _dev(indices)
    s["pool"], s["scales"] = _make_pool(c, g, pool)
    return s


def prepare(case, seed):
    s, c = _inputs(case, seed), case
    if own and c["op"] == "decode":  # the plan that a program makes once for all layers of a step
        from paged_kv_decode_23_gb300 import BatchDecodePagedKV
        dec = BatchDecodePagedKV(torch.empty(128 << 20, dtype=torch.uint8, device="cuda"), c["layout"])
        dec.plan(s["host_indptr"], s["indices"], s["last"], c["hq"], c["hkv"], c["d"], c["page"],
                 window_left=c["window"], logits_soft_cap=c["cap"] or None,
                 q_data_type=DT[c["dtype"]], kv_data_type="e2m1")
        s["plan"] = dec
    return s


# ------------------------------------------------------------------------------------ plain forms
def _power(e):
    """2^e in fp64 for whole e in [-16, 16], exactly (a power function may be off by a rounding)."""
    return torch.tensor([2.0 ** i for i in range(-16, 17)], dtype=torch.float64, device=e.device)[e + 16]


def _over(x, scale):
    """x / scale, rounded once (torch multiplies by a number's reciprocal instead)."""
    return x / torch.full_like(x, scale)


def _to_e4m3(x):
    """Nearest e4m3 value (ties to even) of fp64 x, at most 448."""
    step = _power(torch.frexp(x)[1].clamp(-5, 10) - 4)
    return ((x / step).round() * step).clamp(-448.0, 448.0)


def _to_e2m1(x):
    """Nearest e2m1 value (ties to even) of fp64 x, at most 6."""
    step = _power(torch.frexp(x)[1].clamp(1, 4) - 2)
    return ((x / step).round() * step).clamp(-6.0, 6.0)


def _pack(v):
    """Two e2m1 values a byte, the first in the low half."""
    place = torch.tensor([0, 1, 2, 3, 4, 0, 5, 0, 6, 0, 0, 0, 7], dtype=torch.uint8, device=v.device)
    codes = place[(2 * v.abs()).int()] | ((v < 0).to(torch.uint8) << 3)
    return codes[..., 0::2] | (codes[..., 1::2] << 4)


def _unpack(data, scales, dtype=torch.float32):
    both = torch.tensor(E2M1 + tuple(-x for x in E2M1), dtype=dtype, device=data.device)
    byte = torch.arange(256, device=data.device)
    pairs = torch.stack([both[byte & 15], both[byte >> 4]], dim=1)
    v = pairs[data.int()].flatten(-2)
    return (v.unflatten(-1, (-1, 16)) * scales.to(dtype).unsqueeze(-1)).flatten(-2)


def _where(s, n):
    """(page, slot) of the first n token rows."""
    b, pos = s["batch_indices"][:n].long(), s["positions"][:n].long()
    page = s["case"]["page"]
    return s["indices"][s["indptr"][b].long() + pos // page].long(), pos % page


def _put(s, pool, kv, page, slot, x):
    if s["case"]["layout"] == "NHD":
        pool[page, kv, slot] = x
    else:
        pool[page, kv, :, slot] = x


def _get(s, pool, kv, page, slot):
    return pool[page, kv, slot] if s["case"]["layout"] == "NHD" else pool[page, kv, :, slot]


def _norm_rotate(s, x, weight, n):
    c = s["case"]
    if c["norm"]:
        x = x * torch.rsqrt(x.square().mean(-1, keepdim=True) + EPS) * weight.to(x.dtype)
    r = c["rotary"]
    if r:
        cs = s["cos_sin"][s["positions"][:n].long()].to(x.dtype).unsqueeze(1)
        cos, sin = cs[..., :r // 2], cs[..., r // 2:]
        if c["interleaved"]:
            a, b = x[..., 0:r:2], x[..., 1:r:2]
            turned = torch.stack([a * cos - b * sin, b * cos + a * sin], dim=-1).flatten(-2)
        else:
            a, b = x[..., :r // 2], x[..., r // 2:r]
            turned = torch.cat([a * cos - b * sin, b * cos + a * sin], dim=-1)
        x = torch.cat([turned, x[..., r:]], dim=-1)
    return x


def _plain_append(s):
    c, n = s["case"], s["tokens"]
    exactly = torch.float64 if c["kv"] in ("e4m3", "e2m1") else torch.float32  # codes have borders
    s["q_out"][:n] = _norm_rotate(s, s["q"][:n].float(), s.get("q_weight"), n).to(s["q_out"].dtype)
    k = _norm_rotate(s, s["k"][:n].to(exactly), s.get("k_weight"), n)
    v = s["v"][:n].to(exactly)
    page, slot = _where(s, n)
    for kv, x in ((0, k), (1, v)):
        if c["kv"] == "e2m1":
            scale = s["v_scale" if kv else "k_scale"]
            x = x.unflatten(-1, (-1, 16))
            sf = _to_e4m3(_over(x.abs().amax(-1), 6.0 * scale))
            by = (sf * scale).unsqueeze(-1)
            x = _to_e2m1(torch.where(by > 0, x / by, 0.0)).flatten(-2)
            _put(s, s["pool"], kv, page, slot, _pack(x))
            _put(s, s["scales"], kv, page, slot, sf.to(torch.float8_e4m3fn))
        elif c["kv"] == "e4m3":
            x = _to_e4m3(_over(x, s["v_scale" if kv else "k_scale"]))
            _put(s, s["pool"], kv, page, slot, x.to(torch.float8_e4m3fn))
        else:
            _put(s, s["pool"], kv, page, slot, x.to(s["pool"].dtype))
    if c["kv"] == "e2m1":
        return {"q": s["q_out"], "k": _read(s, 0, n, torch.bfloat16), "v": _read(s, 1, n, torch.bfloat16)}
    return {"q": s["q_out"], "cache": s["pool"]}


def _read(s, kv, n, dtype):
    """The first n token rows out of the cache, times their scale."""
    page, slot = _where(s, n)
    x = _get(s, s["pool"], kv, page, slot)
    x = _unpack(x, _get(s, s["scales"], kv, page, slot)) if s["scales"] is not None else x.float()
    return (x * s.get("v_scale" if kv else "k_scale", 1.0)).to(dtype)


def _plain_decode(s):
    c = s["case"]
    b, group, tokens = c["batch"], c["hq"] // c["hkv"], s["table"].shape[1] * c["page"]
    data, scales = s["pool"][s["table"]], s["scales"][s["table"]]  # [batch, pages, 2, ...]
    kv = []
    for i in range(2):
        x = _unpack(data[:, :, i], scales[:, :, i])
        x = x.transpose(2, 3) if c["layout"] == "NHD" else x  # [batch, pages, hkv, page, d]
        kv.append(x.transpose(1, 2).reshape(b, c["hkv"], tokens, c["d"]))
    q = s["q"].float().view(b, c["hkv"], group, c["d"])
    x = torch.matmul(q, kv[0].transpose(2, 3)) * (s["k_scale"] / math.sqrt(c["d"]))
    if c["cap"]:
        x = c["cap"] * torch.tanh(x / c["cap"])
    t = torch.arange(tokens, device="cuda")
    n = s["dev_lens"].unsqueeze(1)
    seen = t < n
    if c["window"] >= 0:
        seen = seen & (t >= n - 1 - c["window"])
    x = torch.where(seen[:, None, None, :], x, -math.inf)
    top = x.amax(-1, keepdim=True)
    p = torch.exp(x - top)
    total = p.sum(-1, keepdim=True)
    o = torch.matmul(p, kv[1]) / total * s["v_scale"]
    lse = (top + torch.log(total)).view(b, c["hq"])
    return {"o": o.view(b, c["hq"], c["d"]).to(DT[c["dtype"]]), "lse": lse}


def _plain_gather(s):
    n = s["tokens"]
    for i, out in ((0, s["k_out"]), (1, s["v_out"])):
        out[:n] = _read(s, i, n, out.dtype)
    return {"k": s["k_out"], "v": s["v_out"]}


def _plain_copy(s):
    for pool in s["pools"]:
        pool[s["dev_dst"]] = pool[s["dev_src"]]
    return s["pools"]


# ------------------------------------------------------------------------------------ own calls
def _own_append(s):
    from paged_kv_decode_23_gb300 import append_paged_kv, gather_paged_kv
    c = s["case"]
    append_paged_kv(s["q"], s["k"], s["v"], s["batch_indices"], s["positions"], s["pool"],
                    s["indptr"], s["indices"], kv_layout=c["layout"], q_weight=s.get("q_weight"),
                    k_weight=s.get("k_weight"), eps=EPS, cos_sin_cache=s.get("cos_sin"),
                    interleaved=c["interleaved"], kv_block_scales=s["scales"],
                    k_scale=s.get("k_scale"), v_scale=s.get("v_scale"), out=s["q_out"])
    if c["kv"] != "e2m1":
        return {"q": s["q_out"], "cache": s["pool"]}
    n = s["tokens"]  # what the 4-bit cache now holds, as values
    k, v = gather_paged_kv(s["batch_indices"][:n], s["positions"][:n], s["pool"], s["indptr"],
                           s["indices"], kv_layout=c["layout"], kv_block_scales=s["scales"],
                           k_scale=s["k_scale"], v_scale=s["v_scale"], out_dtype=torch.bfloat16)
    return {"q": s["q_out"], "k": k, "v": v}


def _own_decode(s):
    o, lse = s["plan"].run(s["q"], s["pool"], kv_block_scales=s["scales"], k_scale=s["k_scale"],
                           v_scale=s["v_scale"], return_lse=True)
    return {"o": o, "lse": lse}


def _own_gather(s):
    from paged_kv_decode_23_gb300 import gather_paged_kv
    k, v = gather_paged_kv(s["batch_indices"], s["positions"], s["pool"], s["indptr"], s["indices"],
                           kv_layout=s["case"]["layout"], kv_block_scales=s["scales"],
                           k_scale=s.get("k_scale"), v_scale=s.get("v_scale"),
                           out=(s["k_out"], s["v_out"]))
    return {"k": k, "v": v}


def _own_copy(s):
    from paged_kv_decode_23_gb300 import copy_pages
    copy_pages(s["pools"], s["src"], s["dst"])
    return s["pools"]


def run(state):
    op = state["case"]["op"]
    if own:
        return {"append": _own_append, "decode": _own_decode, "gather": _own_gather, "copy": _own_copy}[op](state)
    return {"append": _plain_append, "decode": _plain_decode, "gather": _plain_gather, "copy": _plain_copy}[op](state)


# ------------------------------------------------------------------------------------ exact values
def _nearest(x, grid):
    """Nearest of `grid` (ascending, from 0; neighbours alternate even and odd codes) to |x|, ties
    to the even code, the sign kept."""
    a = x.abs()
    mid = (grid[1:] + grid[:-1]) / 2
    i = torch.searchsorted(mid, a.contiguous())  # mids below |x|
    tie = (i < len(mid)) & (a == mid[i.clamp(max=len(mid) - 1)])
    i = i + (tie & (i % 2 == 1))
    return torch.where(x < 0, -grid[i], grid[i])


def _e4m3_grid():
    e = [m * 2.0 ** -9 for m in range(8)]
    e += [(1 + m / 8) * 2.0 ** p for p in range(-6, 9) for m in range(8)]
    return torch.tensor(e[:-1], dtype=torch.float64, device="cuda")  # 448 is the largest


def _values(data, scales):
    """e2m1 codes times scales, in fp64, without a table of bytes."""
    lo, hi = (data & 15).long(), (data >> 4).long()
    code = torch.stack([lo, hi], dim=-1).flatten(-2)
    e, m = (code >> 1) & 3, (code & 1).double()
    mag = torch.where(e == 0, 0.5 * m, (1 + 0.5 * m) * torch.exp2((e - 1).double()))
    return torch.where(code >= 8, -mag, mag) * scales.double().repeat_interleave(16, dim=-1)


def _exact_rows(c, s, x, weight):
    x = x.double()
    if c["norm"]:
        x = x / torch.sqrt((x * x).sum(-1, keepdim=True) / c["d"] + EPS) * weight.double()
    r = c["rotary"]
    if r:
        table = s["cos_sin"].double()[s["positions"][:x.shape[0]].long()]
        turn = torch.complex(table[:, :r // 2], table[:, r // 2:]).unsqueeze(1)
        first = torch.arange(r // 2, device="cuda") * (2 if c["interleaved"] else 1)
        second = first + (1 if c["interleaved"] else r // 2)
        z = torch.complex(x[..., first], x[..., second]) * turn
        x = x.clone()
        x[..., first], x[..., second] = z.real, z.imag
    return x


def exact(case, seed):
    c, s = case, _inputs(case, seed)
    if c["op"] == "copy":
        return None
    if c["op"] == "append":
        n = s["tokens"]
        q = torch.zeros(s["q_out"].shape, dtype=torch.float64, device="cuda")
        q[:n] = _exact_rows(c, s, s["q"][:n], s.get("q_weight"))
        rows = [_exact_rows(c, s, s["k"][:n], s.get("k_weight")), s["v"][:n].double()]
        scale = (s.get("k_scale", 1.0), s.get("v_scale", 1.0))
        if c["kv"] == "e2m1":
            back = []
            for x, by in zip(rows, scale):
                blocks = x.reshape(*x.shape[:2], -1, 16)
                top = blocks.abs().max(dim=-1, keepdim=True)[0]
                sf = _nearest(torch.div(top, torch.tensor(6 * by).to(top)), _e4m3_grid())
                grid = torch.tensor(E2M1, dtype=torch.float64, device="cuda")
                code = _nearest(blocks / (sf * by).clamp(min=1e-300), grid)
                back.append((code * sf * by).reshape(x.shape))
            return {"q": q, "k": back[0], "v": back[1]}
        if c["kv"] == "e4m3":
            rows = [_nearest(torch.div(x, torch.tensor(by).to(x)), _e4m3_grid()) for x, by in zip(rows, scale)]
        cache = s["pool"].double()
        page, slot = _where(s, n)
        for i, x in enumerate(rows):
            _put(s, cache, i, page, slot, x)
        return {"q": q, "cache": cache}
    if c["op"] == "gather":
        n, got = s["tokens"], {}
        for i, name in ((0, "k"), (1, "v")):
            page, slot = _where(s, n)
            x = _get(s, s["pool"], i, page, slot)
            x = _values(x, _get(s, s["scales"], i, page, slot)) if s["scales"] is not None else x.double()
            got[name] = torch.zeros(s[name + "_out"].shape, dtype=torch.float64, device="cuda")
            got[name][:n] = x * s.get(name + "_scale", 1.0)
        return got
    o = torch.zeros(c["batch"], c["hq"], c["d"], dtype=torch.float64, device="cuda")
    lse = torch.zeros(c["batch"], c["hq"], dtype=torch.float64, device="cuda")
    group = c["hq"] // c["hkv"]
    for i in range(c["batch"]):
        n = int(s["lens"][i])
        first = max(0, n - 1 - c["window"]) if c["window"] >= 0 else 0
        pages = s["table"][i, :-(-n // c["page"])]
        kv = []
        for j in range(2):
            x = _values(s["pool"][pages, j], s["scales"][pages, j])
            x = x if c["layout"] == "NHD" else x.movedim(1, 2)
            kv.append(x.reshape(-1, c["hkv"], c["d"])[first:n].repeat_interleave(group, dim=1))
        x = torch.einsum("hd,thd->ht", s["q"][i].double(), kv[0]) * s["k_scale"] / c["d"] ** 0.5
        x = c["cap"] * torch.tanh(x / c["cap"]) if c["cap"] else x
        lse[i] = torch.logsumexp(x, dim=1)
        o[i] = torch.einsum("ht,thd->hd", torch.exp(x - lse[i][:, None]), kv[1]) * s["v_scale"]
    return {"o": o, "lse": lse}
