"""What is measured of the prompt-path operators of the mixed-format paged KV cache: rotary
positions with several axes, causal attention over packed prompts, branching of cached sequences
(fork, truncate, free) and compaction of the page slabs.  ``run`` computes them in plain torch, or
with ``own`` through the pool's calls."""
import numpy as np
import torch

own = False
PAGE = 16


# ------------------------------------------------------------------ cases
def listed():
    return [
        # one short chat turn of a small model: launch latency counts
        dict(name="prompt_turn", op="prompt", lens="37", Hq=8, Hkv=2, D=128),
        # one step of a serving batch: ragged prompts packed without padding, one empty, one of a token
        dict(name="prompt_packed", op="prompt", lens="700,1,17,2048,129,0,333,64,1500", Hq=32, Hkv=8, D=128),
        # prompts of a small model with 64 channels and a KV head per query head
        dict(name="prompt_d64", op="prompt", lens="1000,513,2047,250,3001", Hq=16, Hkv=16, D=64),
        # a document for the 256-channel layout with 6 query heads per KV head
        dict(name="prompt_d256", op="prompt", lens="8192", Hq=24, Hkv=4, D=256),
        # the longest prompt of the 128-channel layout
        dict(name="prompt_long", op="prompt", lens="16384", Hq=32, Hkv=8, D=128),
        # one decode step of 64 sequences at far positions
        dict(name="rope_step", op="rope", rows=64, Hq=32, Hkv=8, D=128, R=128, axes=1, far=131072, pairs="half"),
        # prompts with images: time, height and width positions, the whole head rotated
        dict(name="rope_images", op="rope", rows=16384, Hq=24, Hkv=4, D=256, R=256, axes=3, far=32768, pairs="half"),
        # half of each head rotated, neighbouring channels paired, an odd number of rows
        dict(name="rope_partial", op="rope", rows=20011, Hq=16, Hkv=4, D=64, R=32, axes=2, far=4096, pairs="next"),
        # four samples from one short cached prompt, some then rolled back by a few tokens
        dict(name="branch_few", op="branch", ctx=1003, at=1003, src=1, per=4, cut=3, window=64, Hkv=2, D=128),
        # parallel sampling over 8 layers' rows of a long cached prompt
        dict(name="branch_layers", op="branch", ctx=32768, at=32759, src=8, per=8, cut=5, window=512, Hkv=4, D=256),
        # holes left by a short sequence are closed, then the sequence is cloned again
        dict(name="defrag_short", op="defrag", ctx=1000, stay=500, window=64, Hkv=2, D=128),
        # the same for a long one: the moved and the copied pages are larger than L2
        dict(name="defrag_long", op="defrag", ctx=262144, stay=4096, window=4096, Hkv=8, D=256),
    ]


def draw(rng):
    def log(lo, hi):
        return int(round(lo * (hi / lo) ** rng.random()))

    op = rng.choice(["prompt", "prompt", "rope", "branch", "defrag"])
    if op == "prompt":
        D, Hkv, g = rng.choice([64, 128, 256]), rng.choice([1, 2, 3, 4, 8]), rng.choice([1, 2, 3, 4, 5, 6, 8])
        lens = [log(1, 4096) for _ in range(rng.randint(1, 12))]
        while Hkv * g * sum(lens) ** 2 * D > 32 * 16384 ** 2 * 128:
            lens.pop()
        return dict(op=op, lens=",".join(map(str, lens)), Hq=Hkv * g, Hkv=Hkv, D=D)
    if op == "rope":
        D, Hkv, g = rng.choice([64, 128, 256]), rng.choice([1, 2, 4, 8]), rng.choice([1, 2, 3, 4, 6, 8])
        R, axes = rng.choice([D, D, D // 2, D // 4]), rng.choice([1, 2, 3])
        rows = min(log(1, 40000), 16384 * 28 * 256 // (Hkv * (g + 1) * D))
        return dict(op=op, rows=rows, Hq=Hkv * g, Hkv=Hkv, D=D, R=R, axes=axes, far=log(64, 1 << 20),
                    pairs=rng.choice(["half", "next"]))
    if op == "branch":
        ctx = log(40, 32768)
        window = min(rng.choice([32, 64, 256, 512]), ctx)
        per = rng.randint(1, 8)
        cut = rng.randint(0, 5)
        at = max(1, ctx - rng.randint(0, 9))
        if (per - 1) * cut > min(window - 26, at - 1):  # a cut stays inside the FP8 window
            cut = 0
        return dict(op=op, ctx=ctx, at=at if at > ctx - window + 16 else ctx, src=rng.randint(1, 8), per=per, cut=cut,
                    window=window, Hkv=rng.choice([1, 2, 4, 8]), D=rng.choice([64, 128, 256]))
    return dict(op=op, ctx=log(100, 131072), stay=log(16, 4096), window=rng.choice([32, 64, 512]),
                Hkv=rng.choice([1, 2, 4, 8]), D=rng.choice([64, 128, 256]))


def _lens(case):
    return [int(x) for x in case["lens"].split(",")]


def _pages(n):
    return -(-n // PAGE)


def _formats(n, window):
    """Formats of the pages of a prefilled sequence of n tokens: page 0, the last ``window`` tokens'
    pages and a partial page are FP8 (0), the others TQ3 (1)."""
    p = np.arange(_pages(n))
    return ((p >= 1) & (PAGE * p + PAGE <= n - window)).astype(np.int64)


def _slot_bytes(case):
    return case["Hkv"] * (32 * case["D"] + 16), case["Hkv"] * 14 * case["D"]


def _cache_lens(case):
    """Contexts of the sequences that the cache of a case starts with."""
    if case["op"] == "branch":
        return [case["ctx"]] * case["src"]
    return [case["ctx"], case["stay"], case["ctx"]]


def _cuts(case):
    return [case["at"] - (i % case["per"]) * case["cut"] for i in range(case["src"] * case["per"])]


def work(case):
    if case["op"] == "prompt":
        n = _lens(case)
        return dict(bytes=4.0 * (case["Hq"] + case["Hkv"]) * case["D"] * sum(n),
                    flops=2.0 * case["Hq"] * case["D"] * sum(x * (x + 1) for x in n))
    if case["op"] == "rope":
        rows, heads = case["rows"], case["Hq"] + case["Hkv"]
        return dict(bytes=4.0 * rows * heads * case["D"] + 4.0 * case["axes"] * rows, flops=3.0 * rows * heads * case["R"])
    b8, b3 = _slot_bytes(case)
    if case["op"] == "branch":
        n, per = case["src"] * case["per"], case["per"]
        pages = _pages(case["at"])
        partial = case["at"] % PAGE != 0
        moved = (case["src"] + n) * b8 * partial
        moved += 2 * b8 * sum(c % PAGE != 0 and c // PAGE < case["at"] // PAGE for c in _cuts(case))
        return dict(bytes=float(moved + 4 * pages * (case["src"] + 2 * n)), flops=0)
    f = _formats(case["ctx"], case["window"])
    n3 = int(f.sum())
    return dict(bytes=4.0 * (n3 * b3 + (len(f) - n3) * b8) + 12.0 * len(f), flops=0)


# ------------------------------------------------------------------ inputs
def prepare(case, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)

    def normal(*shape):
        return torch.randn(shape, generator=g, device="cuda", dtype=torch.float32).to(torch.bfloat16)

    if case["op"] == "prompt":
        n, D = sum(_lens(case)), case["D"]
        s = dict(case, q=normal(n, case["Hq"], D), k=normal(n, case["Hkv"], D), v=normal(n, case["Hkv"], D))
        if own:
            s["pool"] = _pool(case, 1, 1, 1, 1)
        return s
    if case["op"] == "rope":
        rows, D, half = case["rows"], case["D"], case["R"] // 2
        s = dict(case, q=normal(rows, case["Hq"], D), k=normal(rows, case["Hkv"], D))
        s["positions"] = torch.randint(0, case["far"], (case["axes"], rows), generator=g, device="cuda", dtype=torch.int32)
        s["inv_freq"] = torch.tensor([10000.0 ** (-i / half) for i in range(half)], dtype=torch.float32, device="cuda")
        s["axis"] = [i * case["axes"] // half for i in range(half)]  # sections of one axis after another
        if own:
            s["pool"] = _pool(case, 1, 1, 1, 1)
        else:
            s["axis"] = torch.tensor(s["axis"], device="cuda")
        return s

    # a cache: the sequences prefilled in order, room for the branches' pages or for a clone
    lens = _cache_lens(case)
    fmts = [_formats(n, case["window"]) for n in lens]
    n3 = int(sum(f.sum() for f in fmts))
    n8 = sum(len(f) for f in fmts) - n3
    n_dst = case["src"] * case["per"] if case["op"] == "branch" else 0
    n8, n3 = n8 + 2 * n_dst + 3, n3 + 5
    rows, cols = len(lens) + n_dst, max(map(_pages, lens)) + 2
    b8, b3 = _slot_bytes(case)
    slab8 = torch.randint(-2 ** 31, 2 ** 31 - 1, (n8 * b8 // 4,), generator=g, device="cuda", dtype=torch.int32)
    slab3 = torch.randint(-2 ** 31, 2 ** 31 - 1, (n3 * b3 // 4,), generator=g, device="cuda", dtype=torch.int32)
    s = dict(case, turn=0)
    if case["op"] == "branch":
        s["dst"] = [len(lens) + i for i in range(n_dst)]
        s["from"] = [i // case["per"] for i in range(n_dst)]
        s["at_list"] = [case["at"]] * n_dst
        s["cuts"] = _cuts(case)
    if own:
        p = s["pool"] = _pool(case, rows, cols, n8, n3)
        for i, n in enumerate(lens):
            zero = torch.zeros((n, case["Hkv"], case["D"]), dtype=torch.bfloat16, device="cuda")
            p.prefill([i], [n], zero, zero, window=case["window"])
        p.buffers[0][: n8 * b8].copy_(slab8.view(torch.uint8))
        p.buffers[1][: n3 * b3].copy_(slab3.view(torch.uint8))
        s["slabs"] = (p.buffers[0][: n8 * b8].view(torch.int32), p.buffers[1][: n3 * b3].view(torch.int32))
        s["table"] = p.buffers[2][: rows * cols * 4].view(torch.int32).view(rows, cols)
        return s
    table = np.full((rows, cols), -1, np.int64)
    first = [0, 0]
    for i, f in enumerate(fmts):
        for t in (0, 1):
            at = np.nonzero(f == t)[0]
            table[i, at] = (t << 30) + first[t] + np.arange(len(at))
            first[t] += len(at)
    s["table"] = torch.tensor(table, dtype=torch.int32, device="cuda")
    s["slabs"] = (slab8, slab3)
    s["pages"] = (slab8.view(n8, -1), slab3.view(n3, -1))
    s["refs"] = tuple(torch.arange(n, device="cuda").lt(first[t]).int() for t, n in ((0, n8), (1, n3)))
    if case["op"] == "branch":
        for key in ("dst", "from", "at_list", "cuts"):
            s[key] = torch.tensor(s[key], device="cuda")
    return s


def _pool(case, rows, cols, n8, n3):
    from mixed_format_paged_mkv_b200 import Pool
    return Pool(case["Hkv"], case["D"], rows, cols, n8, n3)


# ------------------------------------------------------------------ one pass
def run(s):
    if own:
        p = s["pool"]
        if s["op"] == "prompt":
            return p.prompt_attention(s["q"], s["k"], s["v"], _lens(s))
        if s["op"] == "rope":
            return p.rope(s["q"], s["k"], s["positions"], s["inv_freq"], axes=s["axis"], interleaved=s["pairs"] == "next")
        if s["op"] == "branch":
            p.free(s["dst"])
            p.fork(s["from"], s["dst"], s["at_list"])
            p.truncate(s["dst"], s["cuts"])
        else:
            old, kept = (0, 2) if s["turn"] % 2 == 0 else (2, 0)
            p.free([old])
            p.compact()
            p.copy(kept, old)
            s["turn"] += 1
        return dict(slabs=s["slabs"], table=s["table"])
    if s["op"] == "prompt":
        return _plain_prompt(s)
    if s["op"] == "rope":
        return _plain_rope(s)
    if s["op"] == "branch":
        _plain_free(s, s["dst"])
        _plain_fork(s)
        _plain_truncate(s)
    else:
        old, kept = (0, 2) if s["turn"] % 2 == 0 else (2, 0)
        _plain_free(s, torch.tensor([old], device="cuda"))
        _plain_compact(s, 0)
        _plain_compact(s, 1)
        _plain_copy(s, kept, old)
        s["turn"] += 1
    return dict(slabs=s["slabs"], table=s["table"])


def _plain_prompt(s):
    q, k, v, Hkv = s["q"].float(), s["k"].float(), s["v"].float(), s["Hkv"]
    T, Hq, D = q.shape
    g = Hq // Hkv
    seq = torch.repeat_interleave(torch.tensor(_lens(s), device="cuda"), output_size=T)
    pos = torch.arange(T, device="cuda")
    hidden = (seq[:, None] != seq[None, :]) | (pos[None, :] > pos[:, None])
    qh = q.view(T, Hkv, g, D).permute(1, 2, 0, 3).reshape(Hkv, g * T, D) * (D ** -0.5)
    x = torch.matmul(qh, k.permute(1, 2, 0))
    x.view(Hkv, g, T, T).masked_fill_(hidden, float("-inf"))
    x -= x.amax(-1, keepdim=True)
    x.exp_()
    out = torch.matmul(x, v.permute(1, 0, 2)) / x.sum(-1, keepdim=True)
    return out.view(Hkv, g, T, D).permute(2, 0, 1, 3).reshape(T, Hq, D).to(torch.bfloat16)


def _plain_rope(s):
    angle = s["positions"][s["axis"]].double().t() * s["inv_freq"].double()
    cos, sin = angle.cos().float()[:, None, :], angle.sin().float()[:, None, :]
    return tuple(_rotate(x.float(), cos, sin, s["R"], s["pairs"]).to(torch.bfloat16) for x in (s["q"], s["k"]))


def _rotate(x, cos, sin, R, pairs):
    y = x.clone()
    a, b = (slice(0, R // 2), slice(R // 2, R)) if pairs == "half" else (slice(0, R, 2), slice(1, R, 2))
    y[..., a] = x[..., a] * cos - x[..., b] * sin
    y[..., b] = x[..., b] * cos + x[..., a] * sin
    return y


def _count(s, entries, by):
    """Adds ``by`` to the reference counts of the pages that table entries (-1: none) name."""
    e = entries.reshape(-1).long()
    for t in (0, 1):
        n = s["refs"][t].numel()
        here = (e >= 0) & (e >> 30 == t)
        s["refs"][t].index_add_(0, torch.where(here, e & ((1 << 30) - 1), 0).clamp_(max=n - 1), here.int() * by)


def _plain_free(s, seqs):
    _count(s, s["table"][seqs], -1)
    s["table"][seqs] = -1


def _cut_rows(s, slots, kept):
    """Zeroes the rows from ``kept`` on in the K and V parts of FP8 pages."""
    D, Hkv = s["D"], s["Hkv"]
    page = s["pages"][0].view(-1, Hkv, 8 * D + 4)
    rows = page[slots][:, :, : 8 * D].view(-1, Hkv, 2, PAGE, D // 4)
    rows *= (torch.arange(PAGE, device="cuda")[None, :] < kept[:, None])[:, None, None, :, None]
    page[slots, :, : 8 * D] = rows.reshape(len(slots), Hkv, 8 * D)


def _plain_fork(s):
    at, table = s["at_list"], s["table"]
    full = at // PAGE
    col = torch.arange(table.shape[1], device="cuda")
    rows = torch.where(col < full[:, None], table[s["from"]], -1)
    _count(s, rows, 1)
    table[s["dst"]] = rows
    if s["at"] % PAGE:  # (every branch of a case is taken at the same length)
        new = (s["refs"][0] == 0).nonzero()[: len(at), 0]
        s["pages"][0][new] = s["pages"][0][table[s["from"], full].long()]
        _cut_rows(s, new, at % PAGE)
        s["refs"][0][new] = 1
        table[s["dst"], full] = new.int()


def _plain_truncate(s):
    cuts, table = s["cuts"], s["table"]
    rows = table[s["dst"]]
    keep = (cuts + PAGE - 1) // PAGE
    col = torch.arange(table.shape[1], device="cuda")
    dropped = torch.where(col < keep[:, None], -1, rows)
    last = (cuts // PAGE).clamp(max=table.shape[1] - 1)
    entry = rows.gather(1, last[:, None])[:, 0].long()
    part = (cuts % PAGE != 0).nonzero()[:, 0]
    entry = entry[part]
    shared = s["refs"][0][entry] > 1
    copied = part[shared]
    new = (s["refs"][0] == 0).nonzero()[: len(copied), 0]
    s["pages"][0][new] = s["pages"][0][entry[shared]]
    s["refs"][0][new] = 1
    s["refs"][0].index_add_(0, entry[shared], torch.full_like(new, -1).int())
    rows = torch.where(col < keep[:, None], rows, -1)
    rows[copied, last[copied]] = new.int()
    table[s["dst"]] = rows
    _cut_rows(s, rows[part, last[part]].long(), cuts[part] % PAGE)
    _count(s, dropped, -1)


def _plain_compact(s, t):
    held = s["refs"][t] > 0
    slot = torch.arange(held.numel(), device="cuda")
    front = slot < held.sum()
    moved, holes = (held & ~front).nonzero()[:, 0], (~held & front).nonzero()[:, 0]
    s["pages"][t][holes] = s["pages"][t][moved]
    s["refs"][t][holes] = s["refs"][t][moved]
    s["refs"][t][moved] = 0
    to = slot.clone()
    to[moved] = holes
    e = s["table"].long()
    here = (e >= 0) & (e >> 30 == t)
    at = torch.where(here, e & ((1 << 30) - 1), 0).clamp_(max=held.numel() - 1)
    s["table"].copy_(torch.where(here, (t << 30) + to[at], e))


def _plain_copy(s, src, dst):
    e = s["table"][src].long()
    for t in (0, 1):
        at = ((e >= 0) & (e >> 30 == t)).nonzero()[:, 0]
        new = (s["refs"][t] == 0).nonzero()[: len(at), 0]
        s["pages"][t][new] = s["pages"][t][e[at] & ((1 << 30) - 1)]
        s["refs"][t][new] = 1
        s["table"][dst, at] = ((t << 30) + new).int()


# ------------------------------------------------------------------ the definitions, in 64 bits
def exact(case, seed):
    if case["op"] == "prompt":
        s = prepare(case, seed)
        q, k, v = s["q"].double(), s["k"].double(), s["v"].double()
        out = torch.zeros_like(q)
        g, first = case["Hq"] // case["Hkv"], 0
        for n in _lens(case):
            for h in range(case["Hq"]):
                kh, vh = k[first:first + n, h // g], v[first:first + n, h // g]
                for a in range(0, n, 4096):  # queries [a, b) see the keys before b
                    b = min(n, a + 4096)
                    w = q[first + a:first + b, h] @ kh[:b].t() / case["D"] ** 0.5
                    w.masked_fill_(torch.ones_like(w, dtype=torch.bool).triu_(a + 1), float("-inf"))
                    out[first + a:first + b, h] = torch.softmax(w, -1) @ vh[:b]
            first += n
        return out
    if case["op"] == "rope":
        s = prepare(case, seed)
        half, out = case["R"] // 2, []
        for x in (s["q"].double(), s["k"].double()):
            y = x.clone()
            for i in range(half):
                axis = i * case["axes"] // half
                turn = torch.polar(torch.ones(case["rows"], dtype=torch.float64, device="cuda"),
                                   s["positions"][axis].double() * s["inv_freq"][i].double())
                a, b = (i, i + half) if case["pairs"] == "half" else (2 * i, 2 * i + 1)
                z = torch.complex(x[:, :, a], x[:, :, b]) * turn[:, None]
                y[:, :, a], y[:, :, b] = z.real, z.imag
            out.append(y)
        return tuple(out)
    return None  # pages are moved whole: there is no computed number
