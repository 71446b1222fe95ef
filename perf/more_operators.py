"""Cases of the operators that keep a paged cache bounded while decoding: what is measured, in plain
torch and through this package's entry points.

  sinks    decode attention over a sliding window and the first tokens of each sequence
  weights  decode attention that also adds every key's softmax weight to a pool of sums
  evict    keep each sequence's first, newest and heaviest tokens, in place
"""
import math

import numpy as np
import torch

own = False

DT = {"bf16": torch.bfloat16, "f16": torch.float16, "e4m3": torch.float8_e4m3fn}
E2M1 = (0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0)


# ------------------------------------------------------------------------------------ cases
def listed():
    return [
        # one chat, long past its window: nothing but latency
        dict(name="sinks one", op="sinks", dtype="bf16", kv="bf16", layout="NHD", hq=32, hkv=8, d=128,
             page=16, batch=1, lo=5000, hi=5000, q_len=1, cap=0.0, window=1023, sinks=4),
        # a decode step of 64 chats, most of them past their window of 2,048
        dict(name="sinks batch", op="sinks", dtype="bf16", kv="bf16", layout="NHD", hq=32, hkv=8, d=128,
             page=16, batch=64, lo=512, hi=16000, q_len=1, cap=0.0, window=2047, sinks=4),
        # few very long sequences, a shared preamble of 100 tokens kept in sight, 8-bit cache
        dict(name="sinks long 8-bit", op="sinks", dtype="bf16", kv="e4m3", layout="HND", hq=32, hkv=8, d=128,
             page=64, batch=8, lo=131072, hi=131072, q_len=1, cap=0.0, window=32767, sinks=100),
        # wide heads, soft cap, 4-bit cache, lengths from one token on
        dict(name="sinks 4-bit", op="sinks", dtype="bf16", kv="e2m1", layout="NHD", hq=16, hkv=2, d=256,
             page=32, batch=128, lo=1, hi=8192, q_len=1, cap=30.0, window=4096, sinks=17),
        # one sequence decodes its next token and its keys' weights are summed
        dict(name="weights one", op="weights", dtype="bf16", kv="bf16", layout="HND", hq=32, hkv=8, d=128,
             page=16, batch=1, lo=777, hi=777, q_len=1, cap=0.0, window=-1, sinks=0),
        # the framework's headline batch
        dict(name="weights batch", op="weights", dtype="bf16", kv="bf16", layout="NHD", hq=32, hkv=8, d=128,
             page=16, batch=64, lo=512, hi=4096, q_len=1, cap=0.0, window=-1, sinks=0),
        # few very long sequences: each is split over the whole GPU
        dict(name="weights long", op="weights", dtype="f16", kv="f16", layout="HND", hq=32, hkv=8, d=128,
             page=64, batch=4, lo=131072, hi=131072, q_len=1, cap=0.0, window=-1, sinks=0),
        # wide heads, 8-bit cache, soft cap, window and sinks at once, lengths from one token on
        dict(name="weights window 8-bit", op="weights", dtype="bf16", kv="e4m3", layout="NHD", hq=16, hkv=2,
             d=256, page=32, batch=128, lo=1, hi=8192, q_len=1, cap=30.0, window=4096, sinks=4),
        # one chat has outgrown its budget by a page
        dict(name="evict one", op="evict", kv="bf16", layout="NHD", hkv=8, d=128, page=16, batch=1, lo=528,
             hi=528, budget=512, sinks=4, recent=64),
        # 64 chats are cut back to their budget after 16 decode steps each
        dict(name="evict steps", op="evict", kv="bf16", layout="NHD", hkv=8, d=128, page=16, batch=64, lo=2049,
             hi=2064, budget=2048, sinks=4, recent=128),
        # long prompts are cut to a budget before decoding starts
        dict(name="evict prompts", op="evict", kv="f16", layout="HND", hkv=8, d=128, page=64, batch=4,
             lo=60000, hi=131072, budget=8192, sinks=4, recent=256),
        # prompts of very different lengths, some of them inside the budget, wide heads in 8 bits
        dict(name="evict ragged 8-bit", op="evict", kv="e4m3", layout="NHD", hkv=2, d=256, page=32, batch=33,
             lo=500, hi=9000, budget=1999, sinks=1, recent=31),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["sinks", "weights", "evict"])
    d = rng.choice([64, 128, 128, 256])
    hkv = rng.choice([1, 2, 3, 4, 8])
    page = rng.choice([8, 16, 32, 64])
    layout = rng.choice(["NHD", "HND"])
    dtype = rng.choice(["bf16", "f16"])
    kv = rng.choice([dtype, "e4m3" if d > 64 else dtype, "e2m1"])
    batch = _log(rng, 1, 128)
    most = 500000 * 8 * 128 // (batch * hkv * d)  # tokens of a sequence, by what the pools may hold
    if op == "evict":
        hi = _log(rng, 2, max(3, min(131072, most)))
        budget = max(1, hi - _log(rng, 1, hi)) if rng.random() < 0.5 else _log(rng, 1, hi)
        sinks = rng.choice([0, 1, 4, budget // 3])
        sinks = min(sinks, budget)
        recent = min(budget - sinks, rng.choice([0, 1, 16, 100, budget // 2]))
        return dict(op=op, kv=kv, layout=layout, hkv=hkv, d=d, page=page, batch=batch,
                    lo=rng.randint(1, hi), hi=hi, budget=budget, sinks=sinks, recent=recent)
    q_len = rng.choice([1, 1, 1, 2, 4])
    hi = _log(rng, 1, max(2, min(131072, most // q_len)))
    bounded = op == "sinks" or rng.random() < 0.3
    return dict(op=op, dtype=dtype, kv=kv, layout=layout, hq=hkv * rng.choice([1, 4, 6, 8, 12]), hkv=hkv, d=d,
                page=page, batch=batch, lo=rng.randint(1, hi), hi=hi, q_len=q_len, cap=rng.choice([0.0, 0.0, 30.0]),
                window=rng.randint(0, hi) if bounded else -1,
                sinks=rng.choice([1, 4, 4, 17, 128, 1000]) if bounded else 0)


def _lens(c):
    return np.rint(np.linspace(c["lo"], c["hi"], c["batch"])).astype(np.int64)


def _row_bytes(c):  # of K alone, one token and kv head
    return {"e2m1": c["d"] // 2 + c["d"] // 16, "e4m3": c["d"]}.get(c["kv"], 2 * c["d"])


def _spans(c, lens):
    """(keys, first key of the window, sinks before it) of every query row, row-major by sequence."""
    back = np.arange(c["q_len"])[::-1]
    n = np.maximum(lens[:, None] - back[None, :], 0).reshape(-1)
    w = np.maximum(n - 1 - c["window"], 0) if c["window"] >= 0 else np.zeros_like(n)
    return n, w, np.minimum(c["sinks"], w)


def work(case):
    c = case
    row = _row_bytes(c)
    if c["op"] == "evict":
        n = _lens(c).astype(np.float64)
        n = n[n > c["budget"]]
        b, s, r = c["budget"], c["sinks"], c["recent"]
        moved = r + (b - s - r) * (n - b) / np.maximum(n - r - s, 1)  # weights have no order
        per_head = 4 * (n - s) + moved * (4 * row + 4) + 4 * (n - b)
        return {"bytes": float(c["hkv"] * (per_head.sum() + 4 * b * c["batch"])), "flops": 0}
    n, w, s = _spans(c, _lens(c))
    rows = n.shape[0]
    attended = int((n - w + s).sum())
    # (the query rows of one sequence see nearly the same keys, which have to be read once)
    once = int((n - w + s).reshape(-1, c["q_len"])[:, -1].sum())
    return {"bytes": once * c["hkv"] * (2 * row + (8 if c["op"] == "weights" else 0))
            + rows * c["hq"] * (4 * c["d"] + 4) + 4 * (once // c["page"] + c["batch"]),
            "flops": 4 * attended * c["hq"] * c["d"]}


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
    if c["kv"] != "e2m1":
        x = torch.empty(_shape(c, pages, c["d"]), dtype=DT[c["kv"]], device="cuda")
        for p in range(0, pages, 4096):
            x[p:p + 4096] = _randn(g, *x[p:p + 4096].shape).to(x.dtype)
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


def _dev(a):
    return torch.from_numpy(np.ascontiguousarray(a)).cuda()


def _inputs(c, seed):
    rng, g = np.random.default_rng(seed), _gen(seed)
    s = {"case": c}
    lens = rng.permutation(_lens(c))
    # an evicted sequence owns the pages of its budget, however short it still is
    pages = -(-(np.maximum(lens, c["budget"]) if c["op"] == "evict" else lens) // c["page"])
    pool = int(1.1 * pages.sum()) + 1
    indptr = np.zeros(len(lens) + 1, dtype=np.int32)
    np.cumsum(pages, out=indptr[1:])
    indices = rng.permutation(pool)[:int(indptr[-1])].astype(np.int32)
    s["lens"] = lens
    s["host_indptr"] = torch.from_numpy(indptr)
    s["last"] = torch.from_numpy(np.where(lens > 0, lens - (pages - 1) * c["page"], 0).astype(np.int32))
    s["indptr"], s["indices"] = _dev(indptr), _dev(indices)
    s["kv_lens"] = _dev(lens.astype(np.int32))
    table = np.zeros((len(lens), int(pages.max())), dtype=np.int64)  # padded, for the plain form
    for i in range(len(lens)):
        table[i, :pages[i]] = indices[indptr[i]:indptr[i + 1]]
    s["table"] = _dev(table)
    s["pool"], s["scales"] = _make_pool(c, g, pool)
    if c["kv"] in ("e4m3", "e2m1") and c["op"] != "evict":
        s["k_scale"], s["v_scale"] = 0.75, 1.25
    if c["op"] != "evict":
        s["q"] = _randn(g, c["batch"] * c["q_len"], c["hq"], c["d"]).to(DT[c["dtype"]])
    if c["op"] == "weights":  # as some steps have left them: a few times what one step adds
        s["weights"] = torch.rand((pool, c["hkv"], c["page"]), generator=g, device="cuda") * (4.0 / c["hi"])
    if c["op"] == "evict":
        # sums of many steps, over some orders of magnitude; slots without a token hold nothing
        w = torch.exp(2.0 * _randn(g, pool, c["hkv"], c["page"])) / c["hi"]
        at = torch.arange(table.shape[1] * c["page"], device="cuda")
        mine = torch.zeros((pool, c["page"]), device="cuda")
        seen = (at < s["kv_lens"].unsqueeze(1)).view(len(lens), -1, c["page"])
        for i in range(len(lens)):
            mine[s["table"][i, :pages[i]]] = seen[i, :pages[i]].float()
        s["given"] = w * mine.unsqueeze(1)
        s["weights"] = s["given"].clone()
    return s


def prepare(case, seed):
    s, c = _inputs(case, seed), case
    if own and c["op"] != "evict":  # the plan that a program makes once for all layers of a step
        from paged_kv_decode_23_gb300 import BatchDecodePagedKV
        dec = BatchDecodePagedKV(torch.empty(640 << 20, dtype=torch.uint8, device="cuda"), c["layout"])
        dec.plan(s["host_indptr"], s["indices"], s["last"], c["hq"], c["hkv"], c["d"], c["page"],
                 window_left=c["window"], logits_soft_cap=c["cap"] or None, q_data_type=DT[c["dtype"]],
                 kv_data_type=DT.get(c["kv"], "e2m1"), q_len_per_req=c["q_len"], num_sink_tokens=c["sinks"],
                 key_weights=c["op"] == "weights")
        s["plan"] = dec
    return s


# ------------------------------------------------------------------------------------ plain forms
def _unpack(data, scales):
    """4-bit codes times their scales, in fp32 (exact)."""
    both = torch.tensor(E2M1 + tuple(-x for x in E2M1), device=data.device)
    byte = torch.arange(256, device=data.device)
    pairs = torch.stack([both[byte & 15], both[byte >> 4]], dim=1)
    v = pairs[data.int()].flatten(-2)
    return (v.unflatten(-1, (-1, 16)) * scales.float().unsqueeze(-1)).flatten(-2)


def _at(c, pool, kv, page, slot):
    """Rows [..., kv heads, width] of K (kv = 0) or V at pages and slots of any shape."""
    if c["layout"] == "NHD":
        return pool[page, kv, slot]
    return pool[page, kv, :, slot]


def _rows(s, kv, page, slot):
    c = s["case"]
    x = _at(c, s["pool"], kv, page, slot)
    return _unpack(x, _at(c, s["scales"], kv, page, slot)) if s["scales"] is not None else x.float()


def _attended(s):
    """Positions of each query row's keys, [rows, most], and which of them count."""
    c = s["case"]
    n = (s["kv_lens"].long().unsqueeze(1) - torch.arange(c["q_len"] - 1, -1, -1, device="cuda")).clamp(min=0).view(-1, 1)
    w = (n - 1 - c["window"]).clamp(min=0) if c["window"] >= 0 else torch.zeros_like(n)
    first = w.clamp(max=c["sinks"])
    most = c["hi"] if c["window"] < 0 else min(c["hi"], c["window"] + 1 + c["sinks"])
    i = torch.arange(most, device="cuda")
    t = torch.where(i < first, i, i - first + w)
    seen = t < n
    return torch.where(seen, t, 0), seen


def _plain_decode(s):
    c = s["case"]
    group = c["hq"] // c["hkv"]
    t, seen = _attended(s)
    rows = t.shape[0]
    page = s["table"].repeat_interleave(c["q_len"], dim=0).gather(1, t // c["page"])
    slot = t % c["page"]
    q = s["q"].float().view(rows, c["hkv"], group, c["d"])
    x = torch.matmul(q, _rows(s, 0, page, slot).permute(0, 2, 3, 1)) * (s.get("k_scale", 1.0) / math.sqrt(c["d"]))
    if c["cap"]:
        x = c["cap"] * torch.tanh(x / c["cap"])
    x = torch.where(seen[:, None, None, :], x, -math.inf)
    top = x.amax(-1, keepdim=True)
    top = torch.where(top == -math.inf, 0.0, top)  # a row without a key
    p = torch.exp(x - top)
    total = p.sum(-1, keepdim=True)
    p = torch.where(total > 0, p / total, 0.0)
    o = torch.matmul(p, _rows(s, 1, page, slot).transpose(1, 2)) * s.get("v_scale", 1.0)
    out = {"o": o.view(rows, c["hq"], c["d"]).to(DT[c["dtype"]]),
           "lse": (top + torch.log(total)).view(rows, c["hq"])}
    if c["op"] == "weights":
        heads = torch.arange(c["hkv"], device="cuda").view(1, -1, 1)
        s["weights"].index_put_((page.unsqueeze(1), heads, slot.unsqueeze(1)), p.sum(2), accumulate=True)
        out["weights"] = s["weights"]
    return out


def _plain_evict(s):
    c = s["case"]
    b, first, new = c["budget"], c["sinks"], c["recent"]
    s["weights"].copy_(s["given"])  # what the steps before have summed up
    n = s["kv_lens"].long().view(-1, 1, 1)
    t = torch.arange(max(c["hi"], b), device="cuda")
    page, slot = s["table"][:, t // c["page"]].unsqueeze(1), (t % c["page"]).view(1, 1, -1)
    heads = torch.arange(c["hkv"], device="cuda").view(1, -1, 1)
    w = s["weights"][page, heads, slot]  # [batch, kv heads, tokens]
    may = (t >= first) & (t < n - new)
    order = torch.sort(torch.where(may, w, -1.0), dim=-1, descending=True, stable=True)[1]
    rank = torch.empty_like(order).scatter_(-1, order, t.expand_as(order))
    chosen = may & (rank < b - first - new) & (n > b)
    stays = (t >= first) & (t < b - new)
    free, moves = stays & ~chosen & (n > b), chosen & (t >= b - new)
    place = torch.where(moves, moves.cumsum(-1) - 1, t.shape[0])
    source = torch.zeros((*w.shape[:2], t.shape[0] + 1), dtype=torch.long, device="cuda")
    source.scatter_(-1, place, t.expand_as(place))
    j = t[:b]
    kept = torch.where(free, source.gather(-1, (free.cumsum(-1) - 1).clamp(min=0)), t)[..., :b]
    kept = torch.where((j >= b - new) & (n > b), j + n - b, kept)
    to, at = (s["table"][:, j // c["page"]].unsqueeze(1), heads, (j % c["page"]).view(1, 1, -1)), \
        (s["table"].unsqueeze(1).expand(-1, c["hkv"], -1).gather(2, kept // c["page"]), heads, kept % c["page"])
    pools = [s["pool"]] if s["scales"] is None else [s["pool"], s["scales"]]
    for x in pools:
        x = x.view(torch.uint8) if x.dtype == DT["e4m3"] else x
        for kv in (0, 1):
            one = x[:, kv] if c["layout"] == "HND" else x[:, kv].transpose(1, 2)  # [pages, kv heads, slots, width]
            one.index_put_(to, one[at])
    moved = s["weights"][at]
    gone = (t >= b) & (t < n)
    # (w - w is 0; what lies behind a short sequence's pages adds 0 to some page)
    s["weights"].index_put_((page, heads, slot), torch.where(gone, -w, 0.0), accumulate=True)
    s["weights"].index_put_(to, moved)
    return _evicted(s, torch.where(j < n, kept, -1).int())


def _evicted(s, kept):
    c = s["case"]
    if s["scales"] is None:
        return {"kept": kept, "weights": s["weights"], "cache": s["pool"]}
    t = torch.arange(c["budget"], device="cuda")
    page, slot = s["table"][:, t // c["page"]], (t % c["page"]).unsqueeze(0)
    return {"kept": kept, "weights": s["weights"], "k": _rows(s, 0, page, slot).to(torch.bfloat16),
            "v": _rows(s, 1, page, slot).to(torch.bfloat16)}


# ------------------------------------------------------------------------------------ own calls
def _own_decode(s):
    out = s["plan"].run(s["q"], s["pool"], kv_block_scales=s["scales"], k_scale=s.get("k_scale"),
                        v_scale=s.get("v_scale"), return_lse=True, key_weights=s.get("weights"))
    if s["case"]["op"] == "weights":
        return {"o": out[0], "lse": out[1], "weights": s["weights"]}
    return {"o": out[0], "lse": out[1]}


def _own_evict(s):
    from paged_kv_decode_23_gb300 import evict_paged_kv, gather_paged_kv
    c = s["case"]
    s["weights"].copy_(s["given"])
    kept = evict_paged_kv(s["pool"], s["weights"], s["kv_lens"], s["indptr"], s["indices"], c["budget"],
                          kv_layout=c["layout"], num_sink_tokens=c["sinks"], num_recent=c["recent"],
                          kv_block_scales=s["scales"], return_kept=True)
    if s["scales"] is None:
        return {"kept": kept, "weights": s["weights"], "cache": s["pool"]}
    b = c["budget"]  # what the 4-bit cache now holds, as values
    seq = torch.arange(c["batch"], dtype=torch.int32, device="cuda").repeat_interleave(b)
    pos = torch.arange(b, dtype=torch.int32, device="cuda").repeat(c["batch"])
    k, v = gather_paged_kv(seq, pos, s["pool"], s["indptr"], s["indices"], kv_layout=c["layout"],
                           kv_block_scales=s["scales"], out_dtype=torch.bfloat16)
    return {"kept": kept, "weights": s["weights"], "k": k.view(c["batch"], b, c["hkv"], c["d"]),
            "v": v.view(c["batch"], b, c["hkv"], c["d"])}


def run(state):
    if state["case"]["op"] == "evict":
        return _own_evict(state) if own else _plain_evict(state)
    return _own_decode(state) if own else _plain_decode(state)


# ------------------------------------------------------------------------------------ exact values
def _values(data, scales):
    """e2m1 codes times scales, in fp64, without a table of bytes."""
    code = torch.stack([(data & 15).long(), (data >> 4).long()], dim=-1).flatten(-2)
    e, m = (code >> 1) & 3, (code & 1).double()
    mag = torch.where(e == 0, 0.5 * m, (1 + 0.5 * m) * torch.exp2((e - 1).double()))
    return torch.where(code >= 8, -mag, mag) * scales.double().repeat_interleave(16, dim=-1)


def _sequence(s, i, kv):
    """K (kv = 0) or V of sequence i's whole pages in fp64: [tokens, kv heads, d]."""
    c = s["case"]
    pages = s["indices"][int(s["host_indptr"][i]):int(s["host_indptr"][i + 1])].long()
    x = s["pool"][pages, kv]
    x = _values(x, s["scales"][pages, kv]) if s["scales"] is not None else x.double()
    return (x if c["layout"] == "NHD" else x.movedim(1, 2)).reshape(-1, c["hkv"], c["d"])


def _exact_decode(c, s):
    rows, group = c["batch"] * c["q_len"], c["hq"] // c["hkv"]
    o = torch.zeros(rows, c["hq"], c["d"], dtype=torch.float64, device="cuda")
    lse = torch.full((rows, c["hq"]), -math.inf, dtype=torch.float64, device="cuda")
    sums = s["weights"].double() if c["op"] == "weights" else None
    for i in range(c["batch"]):
        n = int(s["lens"][i])
        k, v = _sequence(s, i, 0)[:n], _sequence(s, i, 1)[:n]
        pages = s["indices"][int(s["host_indptr"][i]):int(s["host_indptr"][i + 1])].long()
        for j in range(c["q_len"]):
            last, r = n - c["q_len"] + j, i * c["q_len"] + j  # the row's own position
            if last < 0:
                continue
            t = torch.arange(last + 1, device="cuda")
            if c["window"] >= 0:
                t = t[(t >= last - c["window"]) | (t < c["sinks"])]
            x = torch.einsum("hgd,thd->hgt", s["q"][r].double().view(c["hkv"], group, c["d"]), k[t])
            x = x * s.get("k_scale", 1.0) / c["d"] ** 0.5
            x = c["cap"] * torch.tanh(x / c["cap"]) if c["cap"] else x
            z = torch.logsumexp(x, dim=2)
            p = torch.exp(x - z[..., None])
            lse[r] = z.view(-1)
            o[r] = torch.einsum("hgt,thd->hgd", p, v[t]).reshape(c["hq"], c["d"]) * s.get("v_scale", 1.0)
            if sums is not None:
                whole = torch.zeros(len(pages) * c["page"], c["hkv"], dtype=torch.float64, device="cuda")
                whole[t] = p.sum(1).t()
                sums[pages] += whole.view(len(pages), c["page"], c["hkv"]).transpose(1, 2)
    return {"o": o, "lse": lse} if sums is None else {"o": o, "lse": lse, "weights": sums}


def _exact_evict(c, s):
    b, first, new = c["budget"], c["sinks"], c["recent"]
    sums, cache = s["given"].double(), None
    if s["scales"] is None:
        cache = s["pool"].double()
    else:
        k, v = (torch.zeros(c["batch"], b, c["hkv"], c["d"], dtype=torch.float64, device="cuda") for _ in range(2))
    kept = torch.full((c["batch"], c["hkv"], b), -1, dtype=torch.int32, device="cuda")
    for i in range(c["batch"]):
        n = int(s["lens"][i])
        pages = s["indices"][int(s["host_indptr"][i]):int(s["host_indptr"][i + 1])].long()
        w = sums[pages].transpose(0, 1).reshape(c["hkv"], -1).clone()
        full = len(pages) * c["page"]
        src = np.tile(np.arange(full), (c["hkv"], 1))
        host = w.cpu().numpy()
        if n > b:
            for h in range(c["hkv"]):
                heavy = np.lexsort((np.arange(first, n - new), -host[h, first:n - new]))[:b - first - new] + first
                heavy = np.sort(heavy)
                holes = np.setdiff1d(np.arange(first, b - new), heavy)
                src[h, holes] = heavy[heavy >= b - new]
                src[h, b - new:b] = np.arange(n - new, n)
        at = torch.from_numpy(src).cuda()
        w = w.gather(1, at)
        if n > b:
            w[:, b:n] = 0
        sums[pages] = w.view(c["hkv"], len(pages), c["page"]).transpose(0, 1)
        kept[i, :, :min(n, b)] = at[:, :min(n, b)].int()
        for kv in (0, 1):
            x = _sequence(s, i, kv).transpose(0, 1)  # [kv heads, tokens, d]
            x = x.gather(1, at[:, :b].unsqueeze(-1).expand(-1, -1, c["d"]))
            if cache is None:
                (v if kv else k)[i] = x.transpose(0, 1)
                continue
            page, slot = pages[torch.arange(b, device="cuda") // c["page"]], torch.arange(b, device="cuda") % c["page"]
            if c["layout"] == "NHD":
                cache[page, kv, slot] = x.transpose(0, 1)
            else:
                cache[page, kv, :, slot] = x.transpose(0, 1)
    out = {"kept": kept, "weights": sums}
    return {**out, "cache": cache} if cache is not None else {**out, "k": k, "v": v}


def exact(case, seed):
    c, s = case, _inputs(case, seed)
    return _exact_evict(c, s) if c["op"] == "evict" else _exact_decode(c, s)
