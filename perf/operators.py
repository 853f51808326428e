"""Measured cases of the sliding-window / dense attention operators and of the cache page operators.

Five kinds of pass (``case["op"]``):

``decode``   attention of one new token per sequence over a paged KV cache, whole context or window + first tokens
``window``   causal sliding-window attention of a prompt, with a few first tokens that stay visible
``train``    the same with its gradients of q, k and v
``branch``   fork sequences of a paged cache, grow the copies, copy the pages they may no longer share, free them
``compact``  move the pages in use to the low end of the pool

``run`` computes them with elementary torch operations, or, where ``own`` is true, with this repository's package.
"""

import math

import torch

own = False

DTYPES = {"f32": torch.float32, "f16": torch.float16, "bf16": torch.bfloat16}
SIZES = {"f32": 4, "f16": 2, "bf16": 2}
CHUNK = 512  # query rows that the plain form takes against one band of keys


def listed():
    return [
        # one sequence of a chat, short context: what a single user waits for at every token
        dict(name="decode one", op="decode", batch=1, lo=1777, hi=1777, heads=32, kv_heads=8, dim=128, dtype="bf16",
             block=64, window=0, sinks=0),
        # an ordinary serving batch with contexts of every length, one query head per KV head
        dict(name="decode ragged", op="decode", batch=16, lo=1, hi=16384, heads=16, kv_heads=16, dim=64, dtype="f16",
             block=64, window=0, sinks=0),
        # the long-context batch: the whole cache is read for one token per sequence
        dict(name="decode long", op="decode", batch=32, lo=32768, hi=65536, heads=32, kv_heads=8, dim=128,
             dtype="bf16", block=64, window=0, sinks=0),
        # a sliding-window layer of the same model family: only the window and the first tokens are read
        dict(name="decode window", op="decode", batch=64, lo=8000, hi=16384, heads=32, kv_heads=4, dim=128,
             dtype="bf16", block=128, window=4096, sinks=64),
        # a small padded batch in fp32, as in a numerics check
        dict(name="window small", op="window", batch=2, seq=777, heads=8, kv_heads=2, dim=64, dtype="f32", window=100,
             sinks=5, padded=True),
        # the 32K prompt of a long-context model's sliding-window layer
        dict(name="window 32k", op="window", batch=1, seq=32768, heads=32, kv_heads=8, dim=128, dtype="bf16",
             window=2048, sinks=64, padded=False),
        # a short fine-tuning batch of odd length
        dict(name="train small", op="train", batch=2, seq=513, heads=8, kv_heads=2, dim=64, dtype="f16", window=128,
             sinks=4, padded=False),
        # a long training sequence
        dict(name="train 16k", op="train", batch=1, seq=16384, heads=32, kv_heads=8, dim=128, dtype="bf16",
             window=1024, sinks=16, padded=False),
        # best-of-four of one request, one layer's pools
        dict(name="branch four", op="branch", parents=1, children=4, lo=1000, hi=1000, grow=1, layers=1, pages=128,
             heads=2, dim=64, block=64),
        # speculative branches of a full serving batch, several layers' pools
        dict(name="branch many", op="branch", parents=16, children=96, lo=2000, hi=16384, grow=5, layers=4,
             pages=4096, heads=8, dim=64, block=64),
        # a small pool after a few requests ended
        dict(name="compact small", op="compact", pages=300, live=0.5, batch=8, layers=1, heads=2, dim=64, block=64),
        # a large pool, half of it free in small holes, several layers
        dict(name="compact large", op="compact", pages=4096, live=0.5, batch=64, layers=4, heads=8, dim=64, block=64),
    ]


def _log(rng, lo, hi):
    """A whole number of [lo, hi], even over its logarithm."""
    return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def _heads(rng):
    kv = rng.choice([1, 2, 4, 8])
    return kv * rng.choice([1, 2, 4, 8]), kv


def _window(rng, longest):
    if rng.random() < 0.25:
        return 0, 0
    return _log(rng, 1, max(2, longest)), rng.choice([0, 0, 1, 4, 7, 64, 100, 128])


def draw(rng):
    op = rng.choice(["decode", "window", "train", "branch", "compact"])
    if op == "decode":
        heads, kv = _heads(rng)
        dim, batch = rng.choice([64, 128]), _log(rng, 1, 64)
        most = max(1, min(65536, (1 << 31) // (batch * kv * dim)))  # the cache stays below the largest listed one's
        hi = _log(rng, 1, most)
        window, sinks = _window(rng, 8192)
        return dict(op=op, batch=batch, lo=rng.choice([1, hi, (hi + 1) // 2]), hi=hi, heads=heads, kv_heads=kv, dim=dim,
                    dtype=rng.choice(["f16", "bf16"]), block=rng.choice([64, 128]), window=window, sinks=sinks)
    if op in ("window", "train"):
        heads, kv = _heads(rng)
        dim, dtype = rng.choice([64, 128]), rng.choice(["f32", "f16", "bf16", "bf16"])
        batch = rng.choice([1, 1, 2, 3, 4])
        seq = _log(rng, 1, 1024 if dtype == "f32" else 16384)
        window, sinks = _window(rng, 2048 if op == "window" else 1024)
        if window == 0:
            seq = min(seq, 2048)
        # rows x heads x band stay below those of the largest listed case of the kind
        most = (1 << 31) if op == "window" else (3 << 28)
        while batch * heads * seq * (min(window or seq, seq) + CHUNK) > most:
            if batch > 1:
                batch -= 1
            else:
                seq = seq * 2 // 3
        return dict(op=op, batch=batch, seq=seq, heads=heads, kv_heads=kv, dim=dim, dtype=dtype, window=window,
                    sinks=sinks, padded=rng.random() < 0.4)
    dim, block = rng.choice([64, 128]), rng.choice([64, 128])
    heads = rng.choice([1, 2, 4])
    if op == "branch":
        parents = _log(rng, 1, 16)
        hi = _log(rng, 1, 16384)
        children, grow = _log(rng, 1, 64), _log(rng, 1, 300)
        pages = parents * -(-hi // block) + children * (-(-grow // block) + 2) + rng.randrange(1, 200)
        return dict(op=op, parents=parents, children=children, lo=rng.choice([1, (hi + 1) // 2, hi]), hi=hi, grow=grow,
                    layers=rng.choice([1, 2]), pages=pages, heads=heads, dim=dim, block=block)
    return dict(op=op, pages=_log(rng, 16, 4096), live=rng.choice([0.1, 0.3, 0.5, 0.7, 0.95]), batch=_log(rng, 1, 64),
                layers=rng.choice([1, 2]), heads=heads, dim=dim, block=block)


# ------------------------------------------------------------------ inputs


def _lengths(lo, hi, n):
    """n lengths spread evenly over [lo, hi] (the same for every seed; their order is the seed's)."""
    return [hi - (hi - lo) * i // max(1, n - 1) if n > 1 else hi for i in range(n)]


def _shuffled(values, gen):
    return torch.tensor(values)[torch.randperm(len(values), generator=gen)]


def _rows_of(case):
    """Lengths of the sequences of a padded batch."""
    s = case["seq"]
    return _lengths(-(-s // 3), s, case["batch"]) if case["padded"] else [s] * case["batch"]


def prepare(case, seed):
    dev = torch.device("cuda")
    cpu = torch.Generator().manual_seed(seed)
    gpu = torch.Generator(device=dev).manual_seed(seed)
    op = case["op"]

    def normal(*shape, dtype):
        return torch.randn(shape, generator=gpu, device=dev, dtype=dtype)

    if op == "decode":
        dt, block, batch = DTYPES[case["dtype"]], case["block"], case["batch"]
        lengths = _shuffled(_lengths(case["lo"], case["hi"], batch), cpu)
        most = -(-case["hi"] // block)
        used = [-(-int(n) // block) for n in lengths]
        ids = torch.randperm(sum(used) + 3, generator=cpu)  # pages in the order of a pool in long use
        table, at = torch.full((batch, most), -1, dtype=torch.int32), 0
        for b, n in enumerate(used):
            table[b, :n] = ids[at:at + n]
            at += n
        shape = (len(ids), block, case["kv_heads"], case["dim"])
        return dict(case=case, q=normal(batch, 1, case["heads"], case["dim"], dtype=dt), k=normal(*shape, dtype=dt),
                    v=normal(*shape, dtype=dt), table=table.to(dev), seqlens=lengths.to(torch.int32).to(dev))
    if op in ("window", "train"):
        dt = DTYPES[case["dtype"]]
        b, s, d = case["batch"], case["seq"], case["dim"]
        st = dict(case=case, q=normal(b, s, case["heads"], d, dtype=dt), k=normal(b, s, case["kv_heads"], d, dtype=dt),
                  v=normal(b, s, case["kv_heads"], d, dtype=dt),
                  seqlens=_shuffled(_rows_of(case), cpu).to(torch.int32).to(dev) if case["padded"] else None)
        if op == "train":
            st["dout"] = normal(b, s, case["heads"], d, dtype=dt)
            for n in "qkv":
                st[n].requires_grad_(True)
        return st
    pages, block = case["pages"], case["block"]
    pools = [normal(pages, block, case["heads"], case["dim"], dtype=torch.bfloat16) for _ in range(2 * case["layers"])]
    ids, refs = torch.randperm(pages, generator=cpu), torch.zeros(pages, dtype=torch.int32)
    if op == "branch":
        lengths = _shuffled(_lengths(case["lo"], case["hi"], case["parents"]), cpu)
        rows = case["parents"] + case["children"]
        table = torch.full((rows, -(-(case["hi"] + case["grow"]) // block)), -1, dtype=torch.int32)
        place = torch.randperm(rows, generator=cpu)
        seqlens, at = torch.zeros(rows, dtype=torch.int32), 0
        for i in range(case["parents"]):
            n = -(-int(lengths[i]) // block)
            table[place[i], :n] = ids[at:at + n]
            seqlens[place[i]] = lengths[i]
            at += n
        refs[ids[:at]] = 1
        dst = place[case["parents"]:]
        src = place[torch.randint(0, case["parents"], (case["children"],), generator=cpu)]
        grow = torch.zeros(rows, dtype=torch.int32)
        grow[dst] = case["grow"]
        return dict(case=case, pools=pools, table=table.to(dev), seqlens=seqlens.to(dev), refs=refs.to(dev),
                    src=src.to(torch.int32).to(dev), dst=dst.to(torch.int32).to(dev), grow=grow.to(dev))
    live, batch = max(1, int(pages * case["live"])), case["batch"]
    used = [live // batch + (1 if i < live % batch else 0) for i in range(batch)]
    table, at = torch.full((batch, max(used) + 2), -1, dtype=torch.int32), 0
    seqlens = torch.zeros(batch, dtype=torch.int32)
    for b, n in enumerate(used):
        table[b, :n] = ids[at:at + n]
        seqlens[b] = max(0, n * block - b % block)
        at += n
    if batch > 1 and used[1]:  # a prefix page that two sequences share
        table[1, 0] = table[0, 0]
    held = torch.bincount(table[table >= 0].long(), minlength=pages)
    return dict(case=case, pools=pools, table=table.to(dev), seqlens=seqlens.to(dev),
                refs=held.to(torch.int32).to(dev))


# ------------------------------------------------------------------ the framework's calls


def _own(st):
    import sparse_hierarchical_attention_mean_b200 as dash

    case = st["case"]
    op = case["op"]
    if op == "decode":
        return dash.window_decode_paged(st["q"], st["k"], st["v"], st["table"], st["seqlens"], window=case["window"],
                                        sinks=case["sinks"], return_lse=True)
    if op == "window":
        return dash.window_fwd(st["q"], st["k"], st["v"], window=case["window"], sinks=case["sinks"],
                               seqlens=st["seqlens"])
    if op == "train":
        out = dash.window_attention(st["q"], st["k"], st["v"], window=case["window"], sinks=case["sinks"],
                                    seqlens=st["seqlens"])
        return (out, *torch.autograd.grad(out, (st["q"], st["k"], st["v"]), st["dout"]))
    if op == "branch":
        table, seqlens, refs = st["table"], st["seqlens"], st["refs"]
        dash.pages_fork(table, seqlens, refs, st["src"], st["dst"], case["block"])
        copy_src, copy_dst = dash.pages_grow(table, seqlens, refs, st["grow"], case["block"])
        dash.pages_copy(st["pools"], copy_src, copy_dst)
        dash.pages_free(table, seqlens, refs, st["dst"], case["block"])
        return dict(copy_src=copy_src, copy_dst=copy_dst, table=table, seqlens=seqlens, refs=refs, pools=st["pools"])
    moved = dash.pages_compact(st["table"], st["seqlens"], st["refs"], case["block"])
    dash.pages_copy(st["pools"], moved["src"], moved["dst"])
    return dict(moved, pools=st["pools"])


# ------------------------------------------------------------------ the plain forms


def _plain_decode(st):
    case = st["case"]
    block, window, sinks = case["block"], case["window"], case["sinks"]
    table, n = st["table"].long(), st["seqlens"].long()
    batch, heads, dim, kv = case["batch"], case["heads"], case["dim"], case["kv_heads"]
    dev = table.device
    if window and sinks + window < table.shape[1] * block:  # only the positions that may be seen
        band = n[:, None] - window + torch.arange(window, device=dev)
        first = torch.arange(sinks, device=dev)[None].expand(batch, -1)
        pos = torch.cat([first, band], 1)
        seen = torch.cat([(first < n[:, None]) & (first < n[:, None] - window), band >= 0], 1)
    else:
        pos = torch.arange(table.shape[1] * block, device=dev)[None].expand(batch, -1)
        seen = pos < n[:, None]
        if window:
            seen = seen & ((pos >= n[:, None] - window) | (pos < sinks))
    pos = pos.clamp(0, table.shape[1] * block - 1)
    page = table.gather(1, pos // block).clamp(min=0)
    k = st["k"][page, pos % block].float().permute(0, 2, 3, 1)  # [B, Hkv, d, N]
    q = st["q"].float().reshape(batch, kv, heads // kv, dim)
    s = torch.matmul(q, k) / math.sqrt(dim)
    del k
    s = torch.where(seen[:, None, None], s, s.new_tensor(-math.inf))
    top = s.amax(-1, keepdim=True)
    p = torch.exp(s - top)
    total = p.sum(-1, keepdim=True)
    v = st["v"][page, pos % block].float().permute(0, 2, 1, 3)
    out = torch.matmul(p, v) / total
    lse = (top + torch.log(total)).reshape(batch, heads)
    return out.reshape(batch, 1, heads, dim).to(st["q"].dtype), lse


def _bands(case, dev):
    """For chunks of CHUNK query rows: the positions of the keys they may see, and which of them each row sees."""
    seq = case["seq"]
    window = min(case["window"] or seq, seq)
    sinks = min(case["sinks"] if case["window"] else 0, seq)
    chunks = -(-seq // CHUNK)
    rows = torch.arange(chunks * CHUNK, device=dev).reshape(chunks, CHUNK, 1)
    band = (torch.arange(chunks, device=dev)[:, None] * CHUNK - window + 1
            + torch.arange(CHUNK + window - 1, device=dev)[None])
    first = torch.arange(sinks, device=dev)[None].expand(chunks, -1)
    pos = torch.cat([first, band], 1)  # [chunks, N]
    seen = torch.cat([first[:, None] <= rows - window,
                      (band[:, None] >= 0) & (band[:, None] <= rows) & (band[:, None] > rows - window)], 2)
    return pos.clamp(0, seq - 1), seen, rows


def _split(x, chunks, kv):
    """[B, S, H, d] -> fp32 [B, chunks, Hkv, (rows x G), d], zero rows at the end."""
    b, s, h, d = x.shape
    x = torch.nn.functional.pad(x.float(), (0, 0, 0, 0, 0, chunks * CHUNK - s))
    return x.reshape(b, chunks, CHUNK, kv, h // kv, d).permute(0, 1, 3, 2, 4, 5).reshape(b, chunks, kv, -1, d)


def _joined(x, seq, heads, dtype):
    b, chunks, kv, rg, d = x.shape
    x = x.reshape(b, chunks, kv, CHUNK, rg // CHUNK, d).permute(0, 1, 3, 2, 4, 5)
    return x.reshape(b, chunks * CHUNK, heads, d)[:, :seq].to(dtype)


def _plain_window(st, grads):
    case = st["case"]
    q, k, v = (st[n].detach() for n in "qkv")
    b, seq, heads, dim = q.shape
    kv = case["kv_heads"]
    pos, seen, rows = _bands(case, q.device)
    chunks = pos.shape[0]
    seen = seen[None].expand(b, -1, -1, -1)
    if st["seqlens"] is not None:
        n = st["seqlens"].long()[:, None, None, None]
        seen = seen & (rows[None] < n) & (pos[None, :, None] < n)
    else:
        seen = seen & (rows[None] < seq)
    seen = seen.repeat_interleave(heads // kv, 2)[:, :, None]  # [B, chunks, 1, rows x G, N]
    qc = _split(q, chunks, kv)
    kc = k[:, pos].float().permute(0, 1, 3, 2, 4)  # [B, chunks, Hkv, N, d]
    vc = v[:, pos].float().permute(0, 1, 3, 2, 4)
    s = torch.matmul(qc, kc.transpose(-1, -2)) / math.sqrt(dim)
    s = torch.where(seen, s, s.new_tensor(-math.inf))
    top = s.amax(-1, keepdim=True)
    top = torch.where(top == -math.inf, torch.zeros_like(top), top)
    p = torch.exp(s - top)
    del s
    total = p.sum(-1, keepdim=True)
    p = p / torch.where(total == 0, torch.ones_like(total), total)
    oc = torch.matmul(p, vc)
    out = _joined(oc, seq, heads, q.dtype)
    if not grads:
        return out
    do = _split(st["dout"], chunks, kv)
    dp = torch.matmul(do, vc.transpose(-1, -2))
    ds = p * (dp - (do * oc).sum(-1, keepdim=True)) / math.sqrt(dim)
    del dp
    dq = _joined(torch.matmul(ds, kc), seq, heads, q.dtype)
    where = pos.reshape(-1)

    def spread(x):  # [B, chunks, Hkv, N, d] added up at the keys' positions
        x = x.permute(0, 1, 3, 2, 4).reshape(b, where.numel(), kv, dim)
        return x.new_zeros(b, seq, kv, dim).index_add_(1, where, x)

    dk = spread(torch.matmul(ds.transpose(-1, -2), qc))
    dv = spread(torch.matmul(p.transpose(-1, -2), do))
    return out, dq, dk.to(q.dtype), dv.to(q.dtype)


def _plain_branch(st):
    block = st["case"]["block"]
    table, seqlens, refs, src, dst = st["table"], st["seqlens"], st["refs"], st["src"].long(), st["dst"].long()
    pages, most = refs.numel(), table.shape[1]
    cols = torch.arange(most, device=table.device)

    def held(rows, lens):  # how often each page is held by these rows
        mine = cols < ((lens + block - 1) // block)[:, None]
        return torch.zeros(pages + 1, dtype=torch.int32, device=table.device).scatter_add_(
            0, torch.where(mine, rows, pages).reshape(-1).long(), torch.ones_like(rows).reshape(-1))[:pages]

    def set_rows(rows, new, lens):
        refs.add_(held(new, lens) - held(table[rows], seqlens[rows]))
        blocks, old = (lens + block - 1) // block, (seqlens[rows] + block - 1) // block
        new = torch.where(cols < blocks[:, None], new, torch.full_like(new, -1))
        table[rows] = torch.where(cols < torch.maximum(blocks, old)[:, None], new, table[rows])
        seqlens[rows] = lens

    set_rows(dst, table[src], seqlens[src])
    # grow: a shared partial page is replaced (all holders but the last in order), then new blocks
    n = st["grow"]
    blocks, after = (seqlens + block - 1) // block, (seqlens + n + block - 1) // block
    partial = (n > 0) & (seqlens % block != 0)
    last = table.gather(1, (blocks - 1).clamp(min=0).long()[:, None])[:, 0].clamp(min=0).long()
    same = (last[:, None] == last[None]) & partial[None]
    before = torch.tril(same, -1).sum(1)
    fresh = partial & (before < refs[last] - 1)
    need = after - blocks + fresh
    start = need.cumsum(0) - need
    lowest = torch.sort((refs != 0).to(torch.int32), stable=True).indices.to(torch.int32)
    copy_dst = torch.where(fresh, lowest[start.clamp(max=pages - 1)], -1)
    copy_src = torch.where(fresh, last.to(torch.int32), -1)
    refs.index_add_(0, last, -fresh.to(torch.int32))
    refs[lowest[:int(need.sum())].long()] = 1
    at = (blocks - 1).clamp(min=0).long()[:, None]
    table.scatter_(1, at, torch.where(fresh[:, None], copy_dst[:, None], table.gather(1, at)))
    want = (start + fresh - blocks)[:, None] + cols
    new = (cols >= blocks[:, None]) & (cols < after[:, None])
    table.copy_(torch.where(new, lowest[want.clamp(0, pages - 1)], table))
    seqlens.add_(n)
    _plain_copy(st["pools"], copy_src, copy_dst)
    set_rows(dst, torch.full_like(table[dst], -1), torch.zeros_like(seqlens[dst]))
    return dict(copy_src=copy_src, copy_dst=copy_dst, table=table, seqlens=seqlens, refs=refs, pools=st["pools"])


def _plain_copy(pools, src, dst):
    some = src >= 0
    src, dst = src[some].long(), dst[some].long()
    for pool in pools:
        pool[dst] = pool[src]


def _plain_compact(st):
    block = st["case"]["block"]
    table, refs = st["table"], st["refs"]
    pages = refs.numel()
    ids = torch.arange(pages, device=refs.device)
    live = refs > 0
    count = live.sum()
    hole, tail = ~live & (ids < count), live & (ids >= count)
    src = torch.sort(torch.where(tail, ids, pages)).values
    dst = torch.sort(torch.where(hole, ids, pages)).values
    moves = tail.sum()
    src = torch.where(ids < moves, src, -1).to(torch.int32)
    dst = torch.where(ids < moves, dst, -1).to(torch.int32)
    to = torch.cat([ids.to(torch.int32), ids.new_zeros(1, dtype=torch.int32)])
    to = to.scatter(0, torch.where(src >= 0, src, pages).long(), dst)
    new_refs = torch.zeros_like(to).scatter(0, torch.where(live, to[:pages], pages).long(), refs)[:pages]
    mine = torch.arange(table.shape[1], device=refs.device) < ((st["seqlens"] + block - 1) // block)[:, None]
    new_table = torch.where(mine, to[table.clamp(min=0).long()], table)
    _plain_copy(st["pools"], src, dst)
    return dict(table=new_table, refs=new_refs, src=src[:pages // 2], dst=dst[:pages // 2],
                info=torch.stack([moves, count]).to(torch.int32), pools=st["pools"])


def run(state):
    if own:
        return _own(state)
    op = state["case"]["op"]
    if op == "decode":
        return _plain_decode(state)
    if op in ("window", "train"):
        return _plain_window(state, op == "train")
    return _plain_branch(state) if op == "branch" else _plain_compact(state)


# ------------------------------------------------------------------ work and exact values


def _pairs(seq, window, sinks):
    """How many (row, key) pairs a causal sequence of this length has."""
    w = min(window or seq, seq)
    band = w * (w + 1) // 2 + (seq - w) * w
    far = max(0, seq - w)  # rows with keys before their window: row w + t - 1 has t of them
    c = min(sinks if window else 0, far)
    return band + c * (c + 1) // 2 + (far - c) * c


def work(case):
    op = case["op"]
    if op == "decode":
        seen = [n if not case["window"] or n <= case["window"] else
                case["window"] + min(case["sinks"], n - case["window"])
                for n in _lengths(case["lo"], case["hi"], case["batch"])]
        rows = case["batch"] * case["heads"] * case["dim"]
        return {"bytes": 2 * (2 * sum(seen) * case["kv_heads"] * case["dim"] + 2 * rows),
                "flops": 4 * sum(seen) * case["heads"] * case["dim"]}
    if op in ("window", "train"):
        pairs = sum(_pairs(n, case["window"], case["sinks"]) for n in _rows_of(case))
        q = case["batch"] * case["seq"] * case["heads"] * case["dim"] * SIZES[case["dtype"]]
        kv = q * case["kv_heads"] // case["heads"]
        train = op == "train"
        return {"bytes": (4 * q + 4 * kv) if train else (2 * q + 2 * kv),
                "flops": (14 if train else 4) * pairs * case["heads"] * case["dim"]}
    page = case["block"] * case["heads"] * case["dim"] * 2 * 2 * case["layers"]
    if op == "branch":
        blocks = -(-case["hi"] // case["block"])
        return {"bytes": 2 * case["children"] * page + 4 * (4 * case["children"] * blocks + case["pages"]), "flops": 0}
    live = max(1, int(case["pages"] * case["live"]))
    moves = live * (case["pages"] - live) // case["pages"]  # expected of a random spread
    return {"bytes": 2 * moves * page + 8 * case["pages"] + 8 * live, "flops": 0}


def _exact_decode(st):
    case = st["case"]
    block, g = case["block"], case["heads"] // case["kv_heads"]
    outs, lses = [], []
    for b, n in enumerate(st["seqlens"].tolist()):
        j = torch.arange(n, device=st["q"].device)
        if case["window"]:
            j = j[(j >= n - case["window"]) | (j < case["sinks"])]
        page = st["table"][b].long()[j // block]
        k, v = (st[x][page, j % block].double().repeat_interleave(g, 1) for x in "kv")  # [n, H, d]
        s = torch.einsum("hd,nhd->hn", st["q"][b, 0].double(), k) / math.sqrt(case["dim"])
        lses.append(torch.logsumexp(s, -1))
        outs.append(torch.einsum("hn,nhd->hd", torch.softmax(s, -1), v)[None])
    return torch.stack(outs), torch.stack(lses)


def _exact_window(st):
    case = st["case"]
    b, seq, heads, dim = st["q"].shape
    g, train = heads // case["kv_heads"], case["op"] == "train"
    q, k, v = (st[n].detach() for n in "qkv")
    out = torch.zeros(q.shape, dtype=torch.float64, device=q.device)
    dq, dk, dv = torch.zeros_like(out), *(torch.zeros(k.shape, dtype=torch.float64, device=q.device) for _ in "kv")
    lens = [seq] * b if st["seqlens"] is None else st["seqlens"].tolist()
    for i, n in enumerate(lens):
        for r0 in range(0, n, 2048):
            r1 = min(n, r0 + 2048)
            row = torch.arange(r0, r1, device=q.device)[:, None]
            key = torch.arange(r1, device=q.device)[None]
            hidden = key > row
            if case["window"]:
                hidden = hidden | ((key <= row - case["window"]) & (key >= case["sinks"]))
            for h in range(heads):
                qq, kk, vv = q[i, r0:r1, h].double(), k[i, :r1, h // g].double(), v[i, :r1, h // g].double()
                p = torch.softmax((qq @ kk.T / math.sqrt(dim)).masked_fill(hidden, -math.inf), -1)
                o = p @ vv
                out[i, r0:r1, h] = o
                if train:
                    do = st["dout"][i, r0:r1, h].double()
                    dv[i, :r1, h // g] += p.T @ do
                    ds = p * (do @ vv.T - (do * o).sum(-1, keepdim=True)) / math.sqrt(dim)
                    dq[i, r0:r1, h] = ds @ kk
                    dk[i, :r1, h // g] += ds.T @ qq
    return (out, dq, dk, dv) if train else out


def _exact_pools(st):
    """The pools after the pass, its copies taken one by one in the order of the definition."""
    refs, table, seqlens = st["refs"].tolist(), st["table"].tolist(), st["seqlens"].tolist()
    block, moves = st["case"]["block"], []
    if st["case"]["op"] == "branch":
        grow = st["grow"].tolist()
        for s, d in zip(st["src"].tolist(), st["dst"].tolist()):
            table[d], seqlens[d] = list(table[s]), seqlens[s]
            for page in table[d][:-(-seqlens[d] // block)]:
                refs[page] += 1
        free = (p for p, r in enumerate(list(refs)) if r == 0)
        for b, n in enumerate(grow):
            if n and seqlens[b] % block:
                page = table[b][seqlens[b] // block]
                if refs[page] > 1:
                    refs[page] -= 1
                    moves.append((page, next(free)))
            if n:
                for _ in range(-(-seqlens[b] // block), -(-(seqlens[b] + n) // block)):
                    next(free)
    else:
        count = sum(r > 0 for r in refs)
        moves = list(zip([p for p in range(count, len(refs)) if refs[p] > 0], [p for p in range(count) if refs[p] == 0]))
    pools = [p.double() for p in st["pools"]]
    if moves:
        src, dst = (torch.tensor(x, device=pools[0].device) for x in zip(*moves))
        for p in pools:
            p[dst] = p[src]
    return dict(pools=pools)


def exact(case, seed):
    st = prepare(case, seed)
    with torch.no_grad():
        if case["op"] == "decode":
            return _exact_decode(st)
        return _exact_window(st) if case["op"] in ("window", "train") else _exact_pools(st)
