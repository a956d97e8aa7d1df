"""Cases and plain forms of the operators for requests that share a prompt: page copies, forks,
resizes and compaction of a paged KV cache, and decode attention that reads a shared prefix once.

``own`` False runs each operator's plain form (elementary torch operations); True makes the calls
of this repository's package. State of the page operators: ``block_table`` int32 [rows, max_blocks],
``seq_lens`` int32 [rows] and ``ref_counts`` int32 [num_blocks] (a page whose count is not positive is
free), here views of one int32 buffer, so that a pass that changes them starts from the same state:
one copy puts the buffer back.
"""
import math
import random

import numpy as np
import torch

own = False

DTYPES = {"bf16": torch.bfloat16, "fp16": torch.float16, "fp32": torch.float32}


# --------------------------------------------------------------------------- cases
def listed():
    return [
        # beam search over a 28-layer model with 2 KV heads: eight diverging beams get their own
        # copy of a page, in every layer
        dict(name="copy_8", op="copy", dtype="bf16", layers=28, num_blocks=256, bs=16, n_kv=2, hd=128, n=8),
        # a tenant's prompt pages duplicated: a thousand pages in every layer
        dict(name="copy_1021", op="copy", dtype="fp16", layers=28, num_blocks=2300, bs=16, n_kv=2, hd=128, n=1021),
        # eight samples of one 1000-token prompt
        dict(name="fork_8", op="fork", rows=16, max_blocks=80, num_blocks=512, bs=16, n=8, parents=1, prompt=1000,
             held=20),
        # beam reorder of 255 rows that continue a 32k prompt
        dict(name="fork_255", op="fork", rows=256, max_blocks=2304, num_blocks=8192, bs=16, n=255, parents=4,
             prompt=32755, held=33000),
        # the first decode step after a fork: 64 rows share a partly filled page, every row grows by one
        # token and gets its own copy of that page in all 28 layers
        dict(name="resize_step_64", op="resize", dtype="bf16", layers=28, rows=64, max_blocks=128, num_blocks=1024,
             bs=16, n_kv=2, hd=128, n=64, prompt=1001, grow=1, freed=0, admit=0),
        # churn of a full server: 100 rows end and give their pages back, 29 new prompts of 2000 tokens
        # come in, the other rows grow by one token
        dict(name="resize_churn", op="resize", dtype="fp16", layers=28, rows=256, max_blocks=256, num_blocks=4096,
             bs=32, n_kv=4, hd=64, n=250, prompt=500, grow=1, freed=100, admit=2000),
        # a small cache of 4 layers, half its pages free
        dict(name="compact_small", op="compact", dtype="fp32", layers=4, rows=8, max_blocks=32, num_blocks=255, bs=8,
             n_kv=2, hd=64, fill=0.5),
        # a 28-layer cache after hours of serving: 40 % of the pages live, anywhere
        dict(name="compact_4096", op="compact", dtype="bf16", layers=28, rows=128, max_blocks=128, num_blocks=4096,
             bs=16, n_kv=2, hd=128, fill=0.4),
        # two samples of a short prompt: latency
        dict(name="attn_2x250", op="attn", dtype="bf16", B=2, n_head=12, n_kv=2, hd=128, bs=16, prefix=250, own=20,
             short=0),
        # a batch of 64 behind an 8k prompt, each up to 512 tokens further
        dict(name="attn_64x8192", op="attn", dtype="bf16", B=64, n_head=12, n_kv=2, hd=128, bs=16, prefix=8192,
             own=512, short=0),
        # odd sizes: 33 requests, a prefix that ends inside a page, rows shorter than the prefix, empty rows
        dict(name="attn_33x5003", op="attn", dtype="fp16", B=33, n_head=32, n_kv=4, hd=64, bs=32, prefix=5003,
             own=333, short=3),
        # 256 samples of a 32k context, each up to 1024 tokens further
        dict(name="attn_256x32768", op="attn", dtype="bf16", B=256, n_head=12, n_kv=2, hd=128, bs=16, prefix=32768,
             own=1024, short=0),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng: random.Random):
    op = rng.choice(["copy", "fork", "resize", "compact", "attn", "attn"])
    dtype = rng.choice(["bf16", "bf16", "fp16", "fp32"])
    heads = dict(bs=rng.choice([8, 16, 32]), n_kv=rng.choice([1, 2, 4, 8]), hd=rng.choice([64, 128]))
    if op == "copy":
        layers, n = rng.randint(1, 28), _log(rng, 1, 300)
        return dict(op=op, dtype=dtype, layers=layers, num_blocks=2 * n + rng.randint(1, 99), n=n, **_fit(heads))
    if op == "fork":
        prompt, bs = _log(rng, 1, 30000), heads["bs"]
        held = _log(rng, 1, 30000)
        n = _log(rng, 2, 255)
        parents = rng.randint(1, 4)
        mb = max(prompt, held) // bs + rng.randint(2, 40)
        return dict(op=op, rows=n + parents + rng.randint(0, 9), max_blocks=mb,
                    num_blocks=max(64, 4 * mb) + rng.randint(0, 999), bs=bs, n=n, parents=parents, prompt=prompt,
                    held=held)
    if op == "resize":
        h = _fit(heads)
        rows = _log(rng, 2, 200)
        prompt = _log(rng, 1, 1500)
        n = rng.randint(max(1, rows // 2), rows)
        freed = rng.choice([0, n // 3, n // 2])
        admit = rng.choice([0, _log(rng, 1, 1500)])
        mb = max(prompt + 200, admit) // h["bs"] + rng.randint(1, 9)
        return dict(op=op, dtype=dtype, layers=rng.randint(1, 12), rows=rows, max_blocks=mb,
                    num_blocks=prompt // h["bs"] + rows * (4 + admit // h["bs"] // 3) + rng.randint(8, 99),
                    n=n, prompt=prompt, grow=rng.choice([1, 1, rng.randint(1, 99)]), freed=freed, admit=admit, **h)
    if op == "compact":
        rows, mb = _log(rng, 1, 128), rng.randint(4, 64)
        fill = rng.uniform(0.05, 0.95)
        nb = int(rows * mb / fill / 1.5) + rng.randint(4, 99)
        return dict(op=op, dtype=dtype, layers=rng.randint(1, 5), rows=rows, max_blocks=mb, num_blocks=min(nb, 4095),
                    fill=fill, **_fit(heads))
    group = rng.choice([1, 2, 4, 6, 7, 8])
    hd = rng.choice([64, 128, 128, 256])
    n_kv = rng.choice([1, 2, 4])
    B = _log(rng, 1, 200)
    most = 2.0e10 if dtype != "fp32" else 4.0e9  # 4 * B * n_head * hd * prefix
    prefix = _log(rng, 16, max(17, min(30000, int(most / (4 * B * group * n_kv * hd)))))
    return dict(op="attn", dtype=dtype, B=B, n_head=group * n_kv, n_kv=n_kv, hd=hd, bs=rng.choice([8, 16, 32]),
                prefix=prefix, own=_log(rng, 1, 600), short=rng.choice([0, 0, B // 7]))


def _fit(h):
    """Head layouts of the drawn page cases: up to 32 KB a page and plane."""
    while h["bs"] * h["n_kv"] * h["hd"] > 8192:
        h = dict(h, n_kv=h["n_kv"] // 2)
    return h


# --------------------------------------------------------------------------- inputs
def _caches(c, g):
    shape = (c["layers"], 2, c["num_blocks"], c["bs"], c["n_kv"], c["hd"])
    return torch.randn(shape, generator=g, device="cuda", dtype=torch.float32).to(DTYPES[c["dtype"]])


def _pages(L, bs):
    return -(-L // bs)


def _admitted(c, i):
    """Whether row i of a resize is a new prompt: every second one of the 57 behind the freed rows."""
    return c["admit"] > 0 and c["freed"] <= i < c["freed"] + 57 and (i - c["freed"]) % 2 == 0


def _meta(table, seq, ref):
    """The three arrays as views of one buffer, and a second buffer with their values."""
    parts = [np.ascontiguousarray(a, dtype=np.int32).reshape(-1) for a in (table, seq, ref)]
    begin = torch.from_numpy(np.concatenate(parts)).cuda()
    buf = begin.clone()
    a, b = parts[0].size, parts[0].size + parts[1].size
    return dict(begin=begin, meta=buf, table=buf[:a].view(table.shape), seq=buf[a:b], ref=buf[b:])


def prepare(case, seed):
    c = case
    g = torch.Generator(device="cuda").manual_seed(seed)
    r = np.random.default_rng(seed)
    st = dict(case=c)

    def ints(a):
        return torch.from_numpy(np.asarray(a, dtype=np.int32)).cuda()

    if c["op"] == "copy":
        perm = r.permutation(c["num_blocks"])
        st.update(caches=_caches(c, g), src=ints(r.choice(perm[c["n"]:], c["n"])), dst=ints(perm[:c["n"]]))
    elif c["op"] == "fork":
        # the parents hold a prompt each (the same pages, last page included); the children hold rows
        # of `held` tokens that share pages among themselves
        R, M, NB, bs, P = c["rows"], c["max_blocks"], c["num_blocks"], c["bs"], c["parents"]
        table = np.full((R, M), -1)
        seq = np.zeros(R, dtype=np.int64)
        perm = r.permutation(NB)
        a, b = _pages(c["prompt"], bs), _pages(c["held"], bs)
        rows = r.permutation(R)[:P + c["n"]]
        if c["n"] + P > R:  # a reorder: every parent but the first is a child as well
            rows = np.concatenate([rows[:P], rows[1:P], rows[P:]])[:P + c["n"]]
        parents, children = rows[:P], rows[P:P + c["n"]]
        for row in children:
            table[row, :b], seq[row] = perm[a:a + b], c["held"]
        for row in parents:
            table[row, :a], seq[row] = perm[:a], c["prompt"]
        ref = np.zeros(NB, dtype=np.int64)
        for row in range(R):
            np.add.at(ref, table[row, :_pages(seq[row], bs)], 1)
        st.update(_meta(table, seq, ref), parents=ints(r.choice(parents, c["n"])), children=ints(children))
        if own:
            import swiglu_rmsnorm_add_gb300 as sra
            st["ws"] = sra.kv_fork_workspace(c["n"], M, "cuda")
    elif c["op"] == "resize":
        # rows that continue one prompt, its partly filled last page shared by those that have not
        # grown yet; row i of the call ends (i < freed), comes in with `admit` tokens where it was
        # empty, or grows
        R, M, NB, bs = c["rows"], c["max_blocks"], c["num_blocks"], c["bs"]
        perm = r.permutation(NB)
        a = _pages(c["prompt"], bs)
        table = np.full((R, M), -1)
        seq = np.zeros(R, dtype=np.int64)
        ref = np.zeros(NB, dtype=np.int64)
        rows = r.permutation(R)[:c["n"]]
        used = a
        lens = np.zeros(c["n"], dtype=np.int64)
        for i, row in enumerate(rows):
            if _admitted(c, i):
                lens[i] = c["admit"]
                continue
            table[row, :a], seq[row] = perm[:a], c["prompt"]
            if i % 3 and i < c["freed"] and used + 2 < NB:  # grown apart from the prompt
                extra = min(2, M - a)
                table[row, a:a + extra] = perm[used:used + extra]
                seq[row], used = (a + extra) * bs, used + extra
            lens[i] = 0 if i < c["freed"] else seq[row] + c["grow"]
        for row in range(R):
            np.add.at(ref, table[row, :_pages(seq[row], bs)], 1)
        order = r.permutation(c["n"])
        st.update(_meta(table, seq, ref), caches=_caches(c, g), rows=ints(rows[order]), lens=ints(lens[order]))
        if own:
            import swiglu_rmsnorm_add_gb300 as sra
            st["ws"] = sra.kv_resize_workspace(c["n"], NB, "cuda")
    elif c["op"] == "compact":
        # rows with pages of their own anywhere in the cache, and a prefix shared by every third row
        R, M, NB, bs = c["rows"], c["max_blocks"], c["num_blocks"], c["bs"]
        perm = r.permutation(NB)
        left = max(1, int(NB * c["fill"]))
        table = np.full((R, M), -1)
        seq = np.zeros(R, dtype=np.int64)
        ref = np.zeros(NB, dtype=np.int64)
        shared = min(left, max(1, M // 4))
        used = shared
        for row in range(R):
            k = shared if row % 3 == 0 else 0
            more = min(int(r.integers(0, M - k + 1)), left - used)
            table[row, :k] = perm[:k]
            table[row, k:k + more] = perm[used:used + more]
            used += more
            if k + more:
                seq[row] = (k + more) * bs - int(r.integers(0, bs))
            np.add.at(ref, table[row, :k + more], 1)
        st.update(_meta(table, seq, ref), caches=_caches(c, g))
        if own:
            import swiglu_rmsnorm_add_gb300 as sra
            st["ws"] = sra.kv_compact_workspace(NB, "cuda")
    else:
        B, bs, P = c["B"], c["bs"], c["prefix"]
        more = r.integers(0, c["own"] + 1, size=B)
        more[0] = c["own"]
        lens = P + more
        if c["short"]:  # some rows end inside the prefix, one has nothing
            pick = r.permutation(B)[:c["short"]]
            lens[pick] = r.integers(0, P, size=c["short"])
            lens[pick[0]] = 0
        M = _pages(P + c["own"], bs)
        shared = P // bs  # whole pages of the prefix; a page that it ends inside is each row's own
        need = [max(0, _pages(int(L), bs) - shared) for L in lens]
        NB = _pages(P, bs) + sum(need) + 3
        perm = r.permutation(NB)
        prefix_table = perm[:_pages(P, bs)]
        table = np.full((B, M), -1)
        table[:, :shared] = prefix_table[:shared]
        used = _pages(P, bs)
        for b in range(B):
            table[b, shared:shared + need[b]] = perm[used:used + need[b]]
            used += need[b]
        shape = (2, NB, bs, c["n_kv"], c["hd"])
        dt = DTYPES[c["dtype"]]
        cache = torch.randn(shape, generator=g, device="cuda", dtype=torch.float32).to(dt)
        q = torch.randn((B, c["n_head"], c["hd"]), generator=g, device="cuda", dtype=torch.float32).to(dt)
        if P % bs:  # a row's own copy of the page that the prefix ends inside holds the prefix's tokens
            src = int(prefix_table[P // bs])
            rows = [int(table[b, shared]) for b in range(B) if need[b]]
            cache[:, rows, :P % bs] = cache[:, src:src + 1, :P % bs]
        st.update(q=q, cache=cache, prefix_table=ints(prefix_table), prefix_len=ints([P]), table=ints(table),
                  seq=ints(lens), scale=1.0 / math.sqrt(c["hd"]), longest=int(lens.max()))
        if own:
            import swiglu_rmsnorm_add_gb300 as sra
            st["ws"] = sra.shared_prefix_workspace(B, c["n_head"], c["n_kv"], c["hd"], len(prefix_table), M, bs, dt,
                                                   "cuda")
    return st


# --------------------------------------------------------------------------- one pass
def run(state):
    return (_run_own if own else _run_plain)(state["case"]["op"], state)


def _run_own(op, s):
    import swiglu_rmsnorm_add_gb300 as sra

    c = s["case"]
    if op == "attn":
        return sra.shared_prefix_attention(s["q"], s["cache"], s["prefix_table"], s["prefix_len"], s["table"],
                                           s["seq"], scale=s["scale"], workspace=s["ws"])
    if op == "copy":
        sra.copy_kv_pages(s["caches"], s["src"], s["dst"])
        return s["caches"]
    s["meta"].copy_(s["begin"])
    if op == "fork":
        sra.fork_kv_rows(s["table"], s["seq"], s["ref"], s["parents"], s["children"], c["bs"], workspace=s["ws"])
        return s["table"], s["seq"], s["ref"]
    if op == "resize":
        pos, slot = sra.resize_kv_rows(s["table"], s["seq"], s["ref"], s["rows"], s["lens"], s["caches"],
                                       workspace=s["ws"])
        return s["table"], s["seq"], s["ref"], pos, slot, s["caches"]
    live = sra.compact_kv_pages(s["table"], s["seq"], s["ref"], s["caches"], workspace=s["ws"])
    return s["table"], s["ref"], live, s["caches"]


def _run_plain(op, s):
    if op == "attn":
        return _attention(s)
    if op == "copy":
        s["caches"][:, :, s["dst"].long()] = s["caches"][:, :, s["src"].long()]
        return s["caches"]
    s["meta"].copy_(s["begin"])
    return {"fork": _fork, "resize": _resize, "compact": _compact}[op](s)


def _fork(s):
    table, seq, ref, bs = s["table"], s["seq"], s["ref"], s["case"]["bs"]
    parents, children = s["parents"].long(), s["children"].long()
    j = torch.arange(table.shape[1], device="cuda")
    taken, former = table[parents], table[children]
    length = seq[parents]
    use = j < ((length + bs - 1) // bs)[:, None]
    drop = j < ((seq[children] + bs - 1) // bs)[:, None]
    gain, loss = taken[use].long(), former[drop].long()
    ref.index_add_(0, gain, torch.ones_like(gain, dtype=torch.int32))
    ref.index_add_(0, loss, -torch.ones_like(loss, dtype=torch.int32))
    table[children] = torch.where(use, taken, -1)
    seq[children] = length
    return table, seq, ref


def _resize(s):
    table, seq, ref, bs = s["table"], s["seq"], s["ref"], s["case"]["bs"]
    rows, new = s["rows"].long(), s["lens"]
    old = seq[rows]
    t = table[rows]
    j = torch.arange(table.shape[1], device="cuda")
    had, want = (old + bs - 1) // bs, (new + bs - 1) // bs
    drop = (j >= want[:, None]) & (j < had[:, None])
    loss = t[drop].long()
    ref.index_add_(0, loss, -torch.ones_like(loss, dtype=torch.int32))
    t = torch.where(drop, -1, t)
    grow = new > old
    last = t.gather(1, (had - 1).clamp(min=0).long()[:, None])[:, 0].long()
    cow = grow & (old % bs != 0) & (ref[last.clamp(min=0)] > 1)
    need = torch.where(grow, want - had + cow, 0)
    upto = torch.cumsum(need, 0)
    free = torch.nonzero(ref <= 0)[:, 0]
    served = upto <= free.numel()
    grow, cow = grow & served, cow & served
    first = upto - need
    # the pages of row i: free[first[i]], free[first[i] + 1], ... for its entries from `begin`
    begin = had - cow.int()
    given = (j >= begin[:, None]) & (j < want[:, None]) & grow[:, None]
    pick = (first[:, None] + j - begin[:, None]).clamp(min=0, max=max(0, free.numel() - 1))
    t = torch.where(given, free[pick.long()].to(torch.int32) if free.numel() else t, t)
    fresh = t[given].long()
    ref[fresh] = 1
    lost = last[cow]
    ref.index_add_(0, lost, -torch.ones_like(lost, dtype=torch.int32))
    table[rows] = t
    length = torch.where(grow | (new < old), new, old)
    seq[rows] = length
    # a shared, partly filled last page: its tokens are copied into the row's own page
    dst, keep = t.gather(1, (had - 1).clamp(min=0).long()[:, None])[:, 0].long(), (old % bs)
    tok = torch.arange(bs, device="cuda")
    which, at = torch.nonzero(cow[:, None] & (tok < keep[:, None]), as_tuple=True)
    s["caches"][:, :, dst[which], at] = s["caches"][:, :, last[which], at]
    end = (length - 1).clamp(min=0).long()
    page = t.gather(1, (end // bs)[:, None])[:, 0].long()
    some = length > 0
    return (table, seq, ref, torch.where(some, end, -1), torch.where(some, page * bs + end % bs, -1), s["caches"])


def _compact(s):
    table, seq, ref, bs = s["table"], s["seq"], s["ref"], s["case"]["bs"]
    live = ref > 0
    n = live.sum()
    page = torch.arange(ref.numel(), device="cuda")
    src, dst = torch.nonzero(live & (page >= n))[:, 0], torch.nonzero(~live & (page < n))[:, 0]
    s["caches"][:, :, dst] = s["caches"][:, :, src]
    page[src] = dst
    ref[dst] = ref[src]
    ref[src] = 0
    use = torch.arange(table.shape[1], device="cuda") < ((seq + bs - 1) // bs)[:, None]
    table.copy_(torch.where(use, page[table.clamp(min=0).long()].to(torch.int32), table))
    return table, ref, n.to(torch.int32).reshape(1), s["caches"]


def _attention(s):
    c = s["case"]
    B, H, KV, D, bs, P = c["B"], c["n_head"], c["n_kv"], c["hd"], c["bs"], c["prefix"]
    q = s["q"].float().view(B, KV, H // KV, D) * s["scale"]
    seq = s["seq"].long()
    t = torch.arange(P, device="cuda")
    k, v = (s["cache"][i, s["prefix_table"].long()[t // bs], t % bs].float() for i in (0, 1))  # [P, KV, D]
    a = torch.matmul(q.permute(1, 0, 2, 3).reshape(KV, -1, D), k.permute(1, 2, 0)).view(KV, B, -1, P)
    parts = [a.masked_fill(~(t < seq[:, None])[None, :, None], -math.inf)]
    more = s["longest"] - P
    if more > 0:
        u = torch.arange(P, P + more, device="cuda")
        own_page = s["table"].long()[:, u // bs].clamp(min=0)
        ok, ov = (s["cache"][i, own_page, u % bs].float() for i in (0, 1))  # [B, more, KV, D]
        e = torch.matmul(q, ok.permute(0, 2, 3, 1)).permute(1, 0, 2, 3)
        parts.append(e.masked_fill(~(u < seq[:, None])[None, :, None], -math.inf))
    top = torch.stack([x.amax(-1) for x in parts]).amax(0)[..., None]
    top = torch.where(top == -math.inf, 0.0, top)
    parts = [torch.exp(x - top) for x in parts]
    den = sum(x.sum(-1) for x in parts)[..., None]
    num = torch.matmul(parts[0].view(KV, -1, P), v.permute(1, 0, 2)).view(KV, B, -1, D)
    if more > 0:
        num = num + torch.matmul(parts[1].permute(1, 0, 2, 3), ov.permute(0, 2, 1, 3)).permute(1, 0, 2, 3)
    out = torch.where(den > 0, num / den, 0.0)
    return out.permute(1, 0, 2, 3).reshape(B, H, D).to(s["q"].dtype)


# --------------------------------------------------------------------------- what a pass cannot do without
def work(case):
    """Bytes and operations that a pass cannot do without. The ragged sizes are the expected ones."""
    c = case
    es = 4 if c.get("dtype") == "fp32" else 2
    if c["op"] == "attn":
        own_tokens = c["B"] * c["own"] / 2
        tok = 2 * c["n_kv"] * c["hd"] * es
        rows = c["B"] * c["n_head"] * c["hd"]
        flops = 4 * rows * (c["prefix"] + c["own"] / 2)
        return {"bytes": int((c["prefix"] + own_tokens) * tok + 2 * rows * es), "flops": int(flops)}
    if c["op"] == "fork":
        # the parents' rows read, the children's rows read and written, the counts of their pages changed
        a, b = _pages(c["prompt"], c["bs"]), _pages(c["held"], c["bs"])
        return {"bytes": 4 * (c["parents"] * a + c["n"] * (b + max(a, b) + 4) + 2 * (a + b)),
                "flops": c["n"] * (a + b)}
    page = 2 * c["layers"] * c["bs"] * c["n_kv"] * c["hd"] * es
    if c["op"] == "copy":
        return {"bytes": 2 * c["n"] * page + 8 * c["n"], "flops": 0}
    if c["op"] == "resize":
        # the freed rows' entries, the new prompts' entries, and a copied page for every row that grows
        new = sum(_admitted(c, i) for i in range(c["n"]))
        grown = c["n"] - c["freed"] - new
        part = page * (c["prompt"] % c["bs"]) // c["bs"]
        entries = c["freed"] * _pages(c["prompt"], c["bs"]) + new * _pages(c["admit"], c["bs"]) + 2 * grown
        return {"bytes": 2 * grown * part + 12 * entries + 4 * c["num_blocks"] + 40 * c["n"],
                "flops": entries + c["num_blocks"]}
    moved = c["num_blocks"] * c["fill"] * (1 - c["fill"])
    return {"bytes": int(2 * moved * page + 8 * c["num_blocks"] + 8 * c["rows"] * c["max_blocks"]),
            "flops": 2 * c["num_blocks"]}


# --------------------------------------------------------------------------- in 64 bits
def exact(case, seed):
    """The attention's outputs in 64 bits, a request at a time; the page operators compute no
    numbers (they move values and count), so theirs is None."""
    if case["op"] != "attn":
        return None
    s = prepare(case, seed)
    c, cache = case, s["cache"]
    out = torch.zeros(c["B"], c["n_head"], c["hd"], dtype=torch.float64, device="cuda")
    shared = s["prefix_table"].tolist()
    t_len = c["prefix"]
    group = c["n_head"] // c["n_kv"]
    for b, (length, row) in enumerate(zip(s["seq"].tolist(), s["table"].tolist())):
        if length == 0:
            continue
        where = [shared[t // c["bs"]] * c["bs"] + t % c["bs"] if t < t_len else row[t // c["bs"]] * c["bs"] + t % c["bs"]
                 for t in range(length)]
        flat = cache.flatten(1, 2)[:, torch.tensor(where, device="cuda")].double()
        for h in range(c["n_kv"]):
            heads = slice(h * group, (h + 1) * group)
            w = torch.softmax(s["q"][b, heads].double() @ flat[0, :, h].T * s["scale"], dim=-1)
            out[b, heads] = w @ flat[1, :, h]
    return out
