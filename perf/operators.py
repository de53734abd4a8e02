"""Linear attention with a decay for each head (prompts and single tokens) and the pages of
its state cache (fork, free, compact): measured cases, plain forms and 64-bit references.

For every sequence and key/value head g (heads h with h // (H / Hk) == g share it):
    S_t = exp(log_decay[g]) S_{t-1} + v_t k_t^T        state [V][K], 32 bits
    o_t[h] = scale * S_t q_t[h]
A cache page is one sequence's state at one point, in the arrays of every layer. A row of the
page table is a sequence: its shared snapshots, then its live page (the last one).
"""
import math
import random

import torch

own = False

CHUNK = 128
TYPES = {"bf16": torch.bfloat16, "fp32": torch.float32}


# --------------------------------------------------------------------------------- cases
def listed():
    return [
        # one short fp32 prompt of the smallest configuration: latency
        prefill("prompt tiny fp32", "fp32", 4, 1, 16, 16, nseq=1, seqlen=256),
        # an ordinary batch of prompts, 32 heads of 128
        prefill("prompt batch 4x4096", "bf16", 32, 1, 128, 128, nseq=4, seqlen=4096, init=True),
        # one long document
        prefill("prompt long 65536", "bf16", 16, 1, 128, 128, nseq=1, seqlen=65536),
        # ragged packed prompts, eight heads of 64 share keys and values of 128 (an empty one among them)
        prefill("prompt packed shared heads", "bf16", 8, 8, 128, 64, nseq=16, lo=0, hi=8192, lens=3, init=True),
        # fp32 prompts of an odd length
        prefill("prompt fp32 3x1537", "fp32", 16, 1, 64, 64, nseq=3, seqlen=1537, init=True),
        # one user's next token: latency
        decode("token 1 sequence", "bf16", 32, 1, 128, 128, rows=1, pages=8, padded=0),
        # a full serving batch, states of 512 MiB
        decode("token 256 sequences", "bf16", 32, 1, 128, 128, rows=256, pages=320, padded=0),
        # an odd fp32 batch padded to a fixed size, shared heads
        decode("token padded shared heads", "fp32", 8, 4, 96, 80, rows=64, pages=96, padded=23),
        # one sequence continues as two
        pages("fork one", "fork", 4, 8, 4, 4, 1, layout=1),
        # parallel samples of 16 prompts, eight layers
        pages("fork 64", "fork", 8, 160, 16, 6, 64, layout=2),
        # a few finished sequences leave a small pool (the tiny configuration's pages)
        pages("compact small pages", "compact", 2, 40, 12, 3, 5, layout=3, nheads=4, headdim=16, ngroups=1, dstate=16),
        # half of the sequences finish, eight layers
        pages("compact half", "compact", 8, 256, 64, 6, 32, layout=4),
    ]


def prefill(name, dtype, kv_heads, share, dk, dv, nseq, seqlen=0, lo=0, hi=0, lens=0, init=False, decay="slopes"):
    return {"name": name, "op": "prefill", "dtype": dtype, "kv_heads": kv_heads, "share": share, "dk": dk, "dv": dv,
            "nseq": nseq, "seqlen": seqlen, "lo": lo, "hi": hi, "lens": lens, "init": init, "decay": decay}


def decode(name, dtype, kv_heads, share, dk, dv, rows, pages, padded, decay="slopes"):
    return {"name": name, "op": "decode", "dtype": dtype, "kv_heads": kv_heads, "share": share, "dk": dk, "dv": dv,
            "rows": rows, "pages": pages, "padded": padded, "decay": decay}


def pages(name, op, layers, n_pages, rows, max_pages, n, layout, nheads=64, headdim=64, ngroups=8, dstate=128):
    return {"name": name, "op": op, "layers": layers, "pages": n_pages, "rows": rows, "max_pages": max_pages, "n": n,
            "layout": layout, "nheads": nheads, "headdim": headdim, "ngroups": ngroups, "dstate": dstate}


def spread(rng, lo, hi):
    """A whole number in [lo, hi], spread over its logarithm."""
    return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["prefill", "prefill", "prefill", "decode", "decode", "fork", "compact"])
    if op in ("fork", "compact"):
        small = rng.random() < 0.4
        size = dict(nheads=rng.choice([1, 2, 4, 6]), headdim=rng.choice([16, 32]), ngroups=1, dstate=rng.choice([16, 32])) \
            if small else dict(nheads=rng.choice([16, 32, 64]), headdim=64, ngroups=2, dstate=rng.choice([64, 128]))
        rows, mp = spread(rng, 2, 48), rng.randint(1, 6)
        n = spread(rng, 1, 48) if op == "fork" else rng.randint(1, max(1, rows * 2 // 3))
        c = pages("", op, rng.randint(1, 8), rows * mp + n + rng.randint(0, 16), rows, mp, n, rng.randrange(1 << 20), **size)
    elif op == "decode":
        rows = spread(rng, 1, 256)
        c = decode("", rng.choice(["bf16", "bf16", "fp32"]), rng.choice([1, 2, 4, 8, 16, 32]), rng.choice([1, 1, 2, 4, 8]),
                   rng.choice([16, 40, 64, 96, 128]), rng.choice([16, 40, 64, 80, 128]), rows, rows + rng.randint(0, 64),
                   rng.randint(0, rows - 1) if rng.random() < 0.4 else 0, rng.choice(["slopes", "slopes", "none"]))
    else:
        dtype = rng.choice(["bf16", "bf16", "bf16", "fp32"])
        hk, share = rng.choice([1, 2, 5, 8, 16, 32]), rng.choice([1, 1, 1, 2, 3, 4, 8])
        dk, dv = rng.choice([16, 40, 64, 96, 128]), rng.choice([16, 48, 64, 120, 128])
        budget = (65536 * 16 * 512 if dtype == "bf16" else 4096 * 16 * 512) // (hk * (share + 1) * (dk + dv))
        top = max(1, min(65536, budget))
        packed = rng.random() < 0.5
        total = spread(rng, min(16, top), top)
        nseq = rng.randint(1, 16)
        if packed:
            lo = rng.choice([0, 1, max(0, total // nseq // 4)])
            c = prefill("", dtype, hk, share, dk, dv, nseq, 0, lo, max(lo + 1, total // nseq), rng.randrange(1 << 20))
        else:
            nseq = min(nseq, 6)
            c = prefill("", dtype, hk, share, dk, dv, nseq, max(1, total // nseq))
        c["init"], c["decay"] = rng.random() < 0.5, rng.choice(["slopes", "slopes", "none"])
    del c["name"]
    return c


def lengths(case):
    if case["seqlen"]:
        return [case["seqlen"]] * case["nseq"]
    r = random.Random(case["lens"])
    got = [r.randint(case["lo"], case["hi"]) for _ in range(case["nseq"])]
    got[-1] = max(1, got[-1])
    return got


# --------------------------------------------------------------------------------- inputs
def rand(seed, stream, *shape, dtype=torch.float32):
    g = torch.Generator(device="cuda").manual_seed(seed * 64 + stream)
    return torch.randn(*shape, generator=g, device="cuda", dtype=torch.float32).to(dtype)


def slopes(case):
    """Per head -2^(-8 (g + 1) / Hk): from forgetting within a few tokens to remembering hundreds; "none" keeps all."""
    h = torch.arange(1, case["kv_heads"] + 1, device="cuda", dtype=torch.float64)
    return (-torch.exp2(-8.0 * h / case["kv_heads"]) * (case["decay"] != "none")).float()


def page_layout(case):
    """The pages of every row before the pass (some rows share their first pages with another's) and the rows of the call."""
    r = random.Random(case["layout"])
    op, rows, mp, n = case["op"], case["rows"], case["max_pages"], case["n"]
    live = rows if op == "compact" else max(1, rows)
    free = list(range(case["pages"]))
    r.shuffle(free)
    keep = n if op == "fork" else 0
    table = []
    for i in range(live):
        want = r.randint(1, mp)
        shared = list(table[i - 1][:min(want, len(table[i - 1])) - 1]) if i and r.random() < 0.3 else []
        want = max(1, min(want - len(shared), len(free) - keep - (live - 1 - i)))
        table.append(shared + [free.pop() for _ in range(want)])
    if op == "fork":
        return table, [r.randrange(live) for _ in range(n)], list(range(live, live + n))
    return table, sorted(r.sample(range(live), n)), None


def page_bytes(case):
    conv = case["nheads"] * case["headdim"] + 2 * case["ngroups"] * case["dstate"]
    return case["layers"] * (case["nheads"] * case["headdim"] * case["dstate"] * 4 + conv * 3 * 2)


def prepare(case, seed):
    op = case["op"]
    if op in ("fork", "compact"):
        return prepare_pages(case, seed)
    hk, h = case["kv_heads"], case["kv_heads"] * case["share"]
    dk, dv, dt = case["dk"], case["dv"], TYPES[case["dtype"]]
    s = {"case": case, "log_decay": slopes(case)}
    if op == "decode":
        rows, n = case["rows"], case["pages"]
        r = random.Random(seed)
        at = r.sample(range(n), rows)
        for i in r.sample(range(rows), case["padded"]):
            at[i] = -1
        s |= {"q": rand(seed, 1, rows, h, dk, dtype=dt), "k": rand(seed, 2, rows, hk, dk, dtype=dt) / math.sqrt(dk),
              "v": rand(seed, 3, rows, hk, dv, dtype=dt), "state": rand(seed, 4, n, hk, dv, dk) * 0.5,
              "pages": torch.tensor(at, dtype=torch.int32, device="cuda"), "o": torch.zeros(rows, h, dv, dtype=dt, device="cuda")}
        return s
    lens = lengths(case)
    total = sum(lens)
    lead = (case["nseq"], case["seqlen"]) if case["seqlen"] else (total,)
    s |= {"q": rand(seed, 1, *lead, h, dk, dtype=dt), "k": rand(seed, 2, *lead, hk, dk, dtype=dt) / math.sqrt(dk),
          "v": rand(seed, 3, *lead, hk, dv, dtype=dt), "init": rand(seed, 4, case["nseq"], hk, dv, dk) * 0.5 if case["init"] else None,
          "cu": None if case["seqlen"] else torch.tensor([sum(lens[:i]) for i in range(len(lens) + 1)], dtype=torch.int32, device="cuda"),
          "longest": max(lens)}
    return s


def prepare_pages(case, seed):
    table, first, second = page_layout(case)
    n, rows = case["pages"], len(table) + (len(second) if second else 0)
    conv = case["nheads"] * case["headdim"] + 2 * case["ngroups"] * case["dstate"]
    refs = torch.zeros(n, dtype=torch.int32)
    tab = torch.full((rows, case["max_pages"]), -1, dtype=torch.int32)
    length, live = torch.zeros(rows, dtype=torch.int32), torch.full((rows,), -1, dtype=torch.int32)
    for i, row in enumerate(table):
        tab[i, :len(row)] = torch.tensor(row, dtype=torch.int32)
        length[i], live[i] = len(row), row[-1]
        refs[row] += 1
    dev = lambda v: v if v is None else torch.tensor(v, dtype=torch.int32, device="cuda")  # noqa: E731
    s = {"case": case, "state": rand(seed, 1, case["layers"], n, case["nheads"], case["headdim"], case["dstate"]),
         "conv": rand(seed, 2, case["layers"], n, conv, 3, dtype=torch.bfloat16),
         "saved": torch.cat([refs, tab.flatten(), length, live]).cuda(), "first": dev(first), "second": dev(second)}
    s["meta"] = s["saved"].clone()
    return s


# --------------------------------------------------------------------------------- one pass
def run(s):
    op = s["case"]["op"]
    if op == "prefill":
        return run_prefill(s)
    if op == "decode":
        return run_decode(s)
    # the table as it stood when the request came in; the pass changes it in place
    s["meta"].copy_(s["saved"])
    return run_fork(s) if op == "fork" else run_compact(s)


def run_prefill(s):
    if own:
        from mamba_ssd_state_02_b200 import ssd
        o, final = ssd.linear_attn_fwd(s["q"], s["k"], s["v"], s["log_decay"], init_state=s["init"], cu_seqlens=s["cu"])
        return {"o": o, "final": final}
    q, k, v, cu = s["q"], s["k"], s["v"], s["cu"]
    dtype, (hk, dk), dv = q.dtype, k.shape[-2:], v.shape[-1]
    share, top = q.shape[-2] // hk, s["longest"]
    padded = -(-top // CHUNK) * CHUNK
    if cu is None:
        nseq, lens = q.shape[0], torch.full((q.shape[0],), q.shape[1], device=q.device)
        lay = lambda t: torch.nn.functional.pad(t.float(), (0, 0, 0, 0, 0, padded - top))  # noqa: E731
    else:
        # sequence b's token t is row cu[b] + t; places past its end hold zeros
        nseq, lens = cu.numel() - 1, (cu[1:] - cu[:-1]).long()
        at = torch.arange(padded, device=q.device)
        there = at[None] < lens[:, None]
        rows = (cu[:-1, None].long() + at[None]).clamp(max=q.shape[0] - 1)
        lay = lambda t: t.float()[rows] * there[:, :, None, None]  # noqa: E731
    n = padded // CHUNK
    qc = lay(q).view(nseq, n, CHUNK, hk, share, dk)
    kc, vc = lay(k).view(nseq, n, CHUNK, hk, dk), lay(v).view(nseq, n, CHUNK, hk, dv)
    g = s["log_decay"].double()
    c = torch.arange(CHUNK, device=q.device)
    power = lambda e: torch.exp(g.view(-1, *[1] * e.dim()) * e.double()).float()  # noqa: E731
    scores = torch.einsum("bnthrk,bnshk->bnhrts", qc, kc)
    scores = scores * (power((c[:, None] - c[None]).clamp(min=0)) * (c[:, None] >= c[None]))[:, None]
    o = torch.einsum("bnhrts,bnshv->bnthrv", scores, vc)
    del scores
    # the state entering chunk i: what the earlier chunks add, and the initial state, decayed
    add = torch.einsum("bnshv,bnshk->bnhvk", vc * power(CHUNK - 1 - c).t()[:, :, None], kc) if n > 1 else None
    chunk = torch.arange(n, device=q.device)
    into = torch.zeros(nseq, n, hk, dv, dk, device=q.device)
    if n > 1:
        between = power(((chunk[:, None] - 1 - chunk[None]) * CHUNK).clamp(min=0)) * (chunk[:, None] > chunk[None])
        into = torch.einsum("hij,bjhvk->bihvk", between, add)
    if s["init"] is not None:
        into = into + power(chunk * CHUNK).t()[None, :, :, None, None] * s["init"][:, None]
    o = o + torch.einsum("bnthrk,bnhvk->bnthrv", qc, into) * power(c + 1).t()[:, :, None, None]
    o = (o * dk ** -0.5).reshape(nseq, padded, hk * share, dv)
    t = torch.arange(padded, device=q.device)
    left = (lens[:, None] - 1 - t[None])
    w = (power(left.clamp(min=0)) * (left >= 0)).permute(1, 2, 0)
    final = torch.einsum("bthv,bthk->bhvk", vc.reshape(nseq, padded, hk, dv) * w[..., None], kc.reshape(nseq, padded, hk, dk))
    if s["init"] is not None:
        final = final + power(lens).t()[:, :, None, None] * s["init"]
    if cu is None:
        return {"o": o[:, :top].to(dtype), "final": final}
    seq = torch.repeat_interleave(torch.arange(nseq, device=q.device), lens, output_size=q.shape[0])
    return {"o": o[seq, torch.arange(q.shape[0], device=q.device) - cu[seq]].to(dtype), "final": final}


def run_decode(s):
    if own:
        from mamba_ssd_state_02_b200 import ssd
        ssd.linear_attn_update(s["state"], s["q"], s["k"], s["v"], s["log_decay"], pages=s["pages"], o=s["o"])
        return {"o": s["o"], "state": s["state"]}
    state, pages_, q = s["state"], s["pages"], s["q"].float()
    rows, h, dk = q.shape
    hk = state.shape[1]
    there = pages_ >= 0
    at = torch.where(there, pages_, 0).long()
    lam = torch.exp(s["log_decay"].double()).float()[:, None, None]
    new = lam * state[at] + s["v"].float()[..., None] * s["k"].float()[:, :, None, :]
    o = torch.einsum("bhvk,bhrk->bhrv", new, q.view(rows, hk, h // hk, dk)).reshape(rows, h, -1) * dk ** -0.5
    s["o"].copy_(torch.where(there[:, None, None], o.to(s["o"].dtype), s["o"]))
    # padded rows have no page and write none
    kept = torch.nonzero(there).flatten()
    state.index_copy_(0, at[kept], new[kept])
    return {"o": s["o"], "state": state}


def pool(s):
    """The framework's handle of the cache, made on the first pass and kept as long as the cache is."""
    if "pool" not in s:
        from mamba_ssd_state_02_b200 import ssd
        rows = s["meta"].numel() - s["case"]["pages"]
        s["pool"] = ssd.PagePool([*s["state"], *s["conv"]], rows // (s["case"]["max_pages"] + 2), s["case"]["max_pages"], meta=s["meta"])
    return s["pool"]


def views(s):
    """refcount, table, length and live page of the pool's metadata."""
    meta, n = s["meta"], s["case"]["pages"]
    rows = (meta.numel() - n) // (s["case"]["max_pages"] + 2)
    refs, tab, length, live = torch.split(meta, [n, rows * s["case"]["max_pages"], rows, rows])
    return refs, tab.view(rows, -1), length, live


def run_fork(s):
    refs, table, length, live = views(s)
    parents, children = s["first"].long(), s["second"].long()
    if own:
        from mamba_ssd_state_02_b200 import ssd
        ssd.pages_fork(pool(s), s["first"], s["second"])
    else:
        # earlier pages are shared, the live one is copied into the lowest free pages, child by child
        n, old = length[parents], live[parents].long()
        new = torch.argsort((refs > 0).int(), stable=True)[:parents.numel()]
        place = torch.arange(table.shape[1], device=table.device)[None]
        shared = place < n[:, None] - 1
        refs.index_add_(0, table[parents].clamp(min=0).flatten().long(), shared.flatten().int())
        refs[new] = 1
        table[children] = torch.where(shared, table[parents], torch.where(place == n[:, None] - 1, new[:, None].int(), -1))
        length[children], live[children] = n, new.int()
        s["state"][:, new] = s["state"][:, old]
        s["conv"][:, new] = s["conv"][:, old]
    return {"state": s["state"], "conv": s["conv"], "refs": refs, "table": table, "length": length, "live": live}


def run_compact(s):
    refs, table, length, live = views(s)
    if own:
        from mamba_ssd_state_02_b200 import ssd
        ssd.pages_free(pool(s), s["first"])
        remap, counts = ssd.pages_compact(pool(s))
    else:
        rows = s["first"].long()
        there = table[rows] >= 0
        refs.index_add_(0, table[rows].clamp(min=0).flatten().long(), -there.flatten().int())
        table[rows], length[rows], live[rows] = -1, 0, -1
        # used pages past the new end move, in order, into the free ones before it
        used, at = refs > 0, torch.arange(refs.numel(), device=refs.device)
        end = used.sum()
        src, dst = torch.nonzero(used & (at >= end)).flatten(), torch.nonzero(~used & (at < end)).flatten()
        remap = torch.where(used, at, -1).int()
        remap[src] = dst.int()
        s["state"][:, dst] = s["state"][:, src]
        s["conv"][:, dst] = s["conv"][:, src]
        refs[dst] = refs[src]
        refs[src] = 0
        table.copy_(torch.where(table >= 0, remap[table.clamp(min=0).long()], -1))
        live.copy_(torch.where(live >= 0, remap[live.clamp(min=0).long()], -1))
        counts = torch.stack([end, end.new_full((), src.numel())]).int()
    return {"state": s["state"], "conv": s["conv"], "refs": refs, "table": table, "length": length, "live": live,
            "remap": remap, "counts": counts}


# --------------------------------------------------------------------------------- what it takes
def work(case):
    op = case["op"]
    if op in ("fork", "compact"):
        table, first, second = page_layout(case)
        if op == "fork":
            moved = len(first)
        else:
            kept = {p for i, row in enumerate(table) if i not in set(first) for p in row}
            moved = sum(p >= len(kept) for p in kept)
        meta = 4 * (case["pages"] + (len(table) + (len(second) if second else 0)) * (case["max_pages"] + 2))
        return {"bytes": 2 * moved * page_bytes(case) + 2 * meta, "flops": 0}
    hk, h, dk, dv = case["kv_heads"], case["kv_heads"] * case["share"], case["dk"], case["dv"]
    size = 2 if case["dtype"] == "bf16" else 4
    if op == "decode":
        tokens = case["rows"] - case["padded"]
        states = 2 * tokens
    else:
        tokens = sum(lengths(case))
        states = case["nseq"] * (2 if case["init"] else 1)
    return {"bytes": tokens * (h + hk) * (dk + dv) * size + states * hk * dk * dv * 4, "flops": 2 * tokens * dk * dv * (h + hk)}


# --------------------------------------------------------------------------------- 64 bits
def exact(case, seed):
    """The recurrence itself, token by token in 64 bits; pages have no computed numbers."""
    op = case["op"]
    if op in ("fork", "compact"):
        return None
    s = prepare(case, seed)
    q, k, v = s["q"].double(), s["k"].double(), s["v"].double()
    hk, dk, dv = case["kv_heads"], case["dk"], case["dv"]
    lam = torch.exp(s["log_decay"].double()).view(1, hk, 1, 1)
    scale = 1.0 / math.sqrt(dk)

    def step(S, qt, kt, vt):
        S = S * lam
        S += vt.unsqueeze(-1) * kt.unsqueeze(-2)
        return S, torch.matmul(qt.unflatten(1, (hk, -1)), S.transpose(-1, -2)).flatten(1, 2) * scale

    if op == "decode":
        o, state = s["o"].double(), s["state"].double()
        on = [i for i, p in enumerate(s["pages"].tolist()) if p >= 0]
        at = [s["pages"].tolist()[i] for i in on]
        state[at], o[on] = step(state[at], q[on], k[on], v[on])
        return {"o": o, "state": state}
    lens = lengths(case)
    S = torch.zeros(case["nseq"], hk, dv, dk, dtype=torch.float64, device="cuda") if s["init"] is None else s["init"].double()
    if case["seqlen"]:
        q, k, v = q.flatten(0, 1), k.flatten(0, 1), v.flatten(0, 1)
    o = torch.empty(q.shape[0], q.shape[1], dv, dtype=torch.float64, device="cuda")
    start = [sum(lens[:i]) for i in range(len(lens))]
    # longest first, so that the sequences that still run are the first ones
    order = sorted(range(len(lens)), key=lambda i: -lens[i])
    begin = torch.tensor([start[i] for i in order], device="cuda")
    S = S[order]
    for t in range(max(lens)):
        alive = sum(n > t for n in lens)
        row = begin[:alive] + t
        S[:alive], o[row] = step(S[:alive], q[row], k[row], v[row])
    final = torch.empty_like(S)
    final[order] = S
    return {"o": o.view(case["nseq"], case["seqlen"], *o.shape[1:]) if case["seqlen"] else o, "final": final}
