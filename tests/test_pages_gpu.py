"""Pages of a state cache: append, fork, free, compact and copy against a plain model of the
pool on the host, metadata and bytes exactly."""
import random

import pytest
import torch

pytestmark = pytest.mark.gpu


class Model:
    """What the documentation says, step by step on the host."""

    def __init__(self, arrays, n_rows, max_pages):
        self.arrays = [t.clone() for t in arrays]
        self.n, self.mp = arrays[0].shape[0], max_pages
        self.refs, self.rows = [0] * self.n, [[] for _ in range(n_rows)]

    def _new(self, k):
        free = [p for p in range(self.n) if self.refs[p] == 0]
        return free[:k] if len(free) >= k else None

    def _copy(self, moves):
        for t in self.arrays:
            old = t.clone()
            for s, d in moves:
                t[d] = old[s]

    def append(self, rows, copy_last):
        rows = [r for r in rows if r != -1]
        new = self._new(len(rows))
        if new is None:
            return False
        moves = []
        for r, p in zip(rows, new):
            if copy_last and self.rows[r]:
                moves.append((self.rows[r][-1], p))
            self.rows[r].append(p)
            self.refs[p] = 1
        self._copy(moves)
        return True

    def fork(self, parents, children):
        todo = [(p, c) for p, c in zip(parents, children) if p != -1 and c != -1]
        new = self._new(sum(bool(self.rows[p]) for p, _ in todo))
        if new is None:
            return False
        moves, new = [], list(new)
        for p, c in todo:
            if self.rows[p]:
                page = new.pop(0)
                moves.append((self.rows[p][-1], page))
                for x in self.rows[p][:-1]:
                    self.refs[x] += 1
                self.refs[page] = 1
                self.rows[c] = self.rows[p][:-1] + [page]
        self._copy(moves)
        return True

    def free(self, rows):
        for r in rows:
            if r != -1:
                for p in self.rows[r]:
                    self.refs[p] -= 1
                self.rows[r] = []

    def compact(self):
        used = sum(x > 0 for x in self.refs)
        src = [p for p in range(used, self.n) if self.refs[p] > 0]
        dst = [p for p in range(used) if self.refs[p] == 0]
        remap = [p if self.refs[p] > 0 else -1 for p in range(self.n)]
        for s, d in zip(src, dst):
            remap[s], self.refs[d], self.refs[s] = d, self.refs[s], 0
        self._copy(list(zip(src, dst)))
        self.rows = [[remap[p] for p in r] for r in self.rows]
        return remap, [used, len(src)]

    def copy(self, src, dst):
        self._copy([(s, d) for s, d in zip(src, dst) if s != -1 and d != -1])

    def same(self, pool):
        assert pool.refcount.tolist() == self.refs
        assert pool.table.tolist() == [r + [-1] * (self.mp - len(r)) for r in self.rows]
        assert pool.length.tolist() == [len(r) for r in self.rows]
        assert pool.live.tolist() == [r[-1] if r else -1 for r in self.rows]
        for got, want in zip(pool.arrays, self.arrays):
            assert torch.equal(got.view(torch.uint8) if got.element_size() > 1 else got,
                               want.view(torch.uint8) if want.element_size() > 1 else want)


def make(dev, n, seed=0, odd=True):
    g = torch.Generator().manual_seed(seed)
    r = lambda *s, d=torch.float32: torch.randn(*s, generator=g).to(d).to(dev)  # noqa: E731
    arrays = [r(n, 4, 64, 32), r(n, 40, 3, d=torch.bfloat16), r(n, 40000)]
    if odd:                                    # 20, 6 and 7 bytes a page; one array off 16-byte alignment
        arrays += [r(n, 5), r(n, 3, d=torch.bfloat16), (torch.rand(n, 7, generator=g) * 255).to(torch.uint8).to(dev),
                   r(n * 8 + 1)[1:].view(n, 8)]
    return arrays


def ints(x, dev):
    return torch.tensor(x, dtype=torch.int32, device=dev)


def both(ssd, dev, n, rows, mp, seed=0):
    arrays = make(dev, n, seed)
    return ssd.PagePool([t.clone() if t.data_ptr() % 16 == 0 else t for t in arrays], rows, mp), Model(arrays, rows, mp)


def test_a_new_pool_is_empty(ssd, cuda_dev):
    pool, model = both(ssd, cuda_dev, 6, 4, 3)
    model.same(pool)
    for op in (lambda: ssd.pages_free(pool, ints([0, 3], cuda_dev)), lambda: ssd.pages_fork(pool, ints([0], cuda_dev), ints([1], cuda_dev)),
               lambda: ssd.pages_append(pool, ints([-1, -1], cuda_dev)), lambda: ssd.pages_append(pool, ints([], cuda_dev))):
        op()
        ssd.device_status()
        model.same(pool)
    remap, counts = ssd.pages_compact(pool)
    assert remap.tolist() == [-1] * 6 and counts.tolist() == [0, 0]
    model.same(pool)


@pytest.mark.parametrize("seed", range(6))
def test_random_histories(ssd, cuda_dev, seed):
    """Sixty random requests, some of them with skipped entries, checked one by one."""
    r = random.Random(seed)
    n, rows, mp = r.choice([(40, 12, 5), (9, 4, 3), (200, 64, 4)])
    pool, model = both(ssd, cuda_dev, n, rows, mp, seed)
    for _ in range(60):
        op = r.choice(["append", "append", "fork", "fork", "free", "compact", "copy"])
        empty = [i for i in range(rows) if not model.rows[i]]
        full = [i for i in range(rows) if model.rows[i]]
        ok = True
        if op == "append":
            pick = r.sample([i for i in range(rows) if len(model.rows[i]) < mp], 0) or \
                [i for i in range(rows) if len(model.rows[i]) < mp and r.random() < 0.3]
            pick = [x if r.random() < 0.9 else -1 for x in pick]
            copy = r.random() < 0.5
            ok = model.append(pick, copy)
            ssd.pages_append(pool, ints(pick, cuda_dev), copy_last=copy)
        elif op == "fork" and full and empty:
            children = r.sample(empty, r.randint(1, len(empty)))
            parents = [r.choice(full) if r.random() < 0.9 else -1 for _ in children]
            ok = model.fork(parents, children)
            ssd.pages_fork(pool, ints(parents, cuda_dev), ints(children, cuda_dev))
        elif op == "free":
            pick = r.sample(range(rows), r.randint(0, max(1, rows // 3)))
            model.free(pick)
            ssd.pages_free(pool, ints(pick, cuda_dev))
        elif op == "compact":
            remap, counts = ssd.pages_compact(pool)
            assert (remap.tolist(), counts.tolist()) == tuple(model.compact())
        elif op == "copy":
            at = r.sample(range(n), r.randint(0, n) // 2 * 2)
            src, dst = at[:len(at) // 2], at[len(at) // 2:]
            src = [src[0] if r.random() < 0.3 else x for x in src]           # one source, several copies
            model.copy(src, dst)
            ssd.pages_copy(pool, ints(src, cuda_dev), ints(dst, cuda_dev))
        if ok:
            ssd.device_status()
        else:
            with pytest.raises(ssd.SSDError, match="NO_PAGES"):
                ssd.device_status()
        model.same(pool)


def test_too_few_pages_changes_nothing(ssd, cuda_dev):
    pool, model = both(ssd, cuda_dev, 4, 6, 2)
    ssd.pages_append(pool, ints([0, 1, 2], cuda_dev))
    model.append([0, 1, 2], False)
    for op in (lambda: ssd.pages_append(pool, ints([3, 4], cuda_dev)), lambda: ssd.pages_fork(pool, ints([0, 1], cuda_dev), ints([3, 4], cuda_dev))):
        op()
        with pytest.raises(ssd.SSDError, match="NO_PAGES"):
            ssd.device_status()
        model.same(pool)
    ssd.pages_fork(pool, ints([1], cuda_dev), ints([5], cuda_dev))           # the last one
    model.fork([1], [5])
    ssd.device_status()
    model.same(pool)


@pytest.mark.parametrize("op", [
    ("append", [0, 0]), ("append", [7]), ("append", [-2]), ("append", [2]),               # twice, range, a full row
    ("free", [1, 1]), ("free", [6]), ("free", [-5]),
    ("fork", [0, 0], [4, 4]), ("fork", [0], [1]), ("fork", [0], [0]), ("fork", [0], [6]), ("fork", [6], [4]),
    ("fork", [0, 3], [3, 4]), ("fork", [-2], [4]),                                         # a child that is a parent
    ("copy", [0, 1], [2, 2]), ("copy", [0, 1], [1, 2]), ("copy", [8], [0]), ("copy", [0], [8]), ("copy", [-3], [0]),
])
def test_bad_requests_change_nothing(ssd, cuda_dev, op):
    pool, model = both(ssd, cuda_dev, 8, 6, 2)
    for _ in range(2):
        ssd.pages_append(pool, ints([0, 2], cuda_dev))
        model.append([0, 2], False)
    ssd.pages_append(pool, ints([1], cuda_dev))
    model.append([1], False)
    ssd.device_status()
    getattr(ssd, "pages_" + op[0])(pool, *[ints(x, cuda_dev) for x in op[1:]])
    with pytest.raises(ssd.SSDError, match="INVALID_ARG"):
        ssd.device_status()
    model.same(pool)


@pytest.mark.parametrize("what", ["length", "page"])
def test_corrupt_metadata_is_not_followed(ssd, cuda_dev, what):
    pool, _ = both(ssd, cuda_dev, 8, 6, 2)
    ssd.pages_append(pool, ints([0, 1], cuda_dev))
    if what == "length":
        pool.length[0] = 1000
    else:
        pool.table[0, 0] = 99
        pool.live[0] = 99
    ssd.device_status()
    meta = pool.meta.clone()
    for op in (lambda: ssd.pages_free(pool, ints([0], cuda_dev)), lambda: ssd.pages_fork(pool, ints([0], cuda_dev), ints([3], cuda_dev)),
               lambda: ssd.pages_append(pool, ints([0], cuda_dev), copy_last=True)):
        op()
        with pytest.raises(ssd.SSDError, match="INVALID_ARG"):
            ssd.device_status()
        assert torch.equal(pool.meta, meta)


def test_a_large_pool(ssd, cuda_dev):
    """More pages and rows than one pass of the deciding block (4096 and 1024), lists of thousands."""
    n, rows, mp = 9001, 3001, 3
    arrays = [torch.arange(n * 4, dtype=torch.int32, device=cuda_dev).view(n, 4)]
    pool, model = ssd.PagePool([arrays[0].clone()], rows, mp), Model([arrays[0].cpu()], rows, mp)
    model.arrays = [arrays[0].clone()]
    r = random.Random(1)
    for copy in (False, True):
        pick = r.sample(range(2000), 1900)
        ssd.pages_append(pool, ints(pick, cuda_dev), copy_last=copy)
        assert model.append(pick, copy)
    model.same(pool)
    parents, children = [r.randrange(2000) for _ in range(1000)], list(range(2000, 3000))
    ssd.pages_fork(pool, ints(parents, cuda_dev), ints(children, cuda_dev))
    assert model.fork(parents, children)
    model.same(pool)
    gone = r.sample(range(3000), 2000)
    ssd.pages_free(pool, ints(gone, cuda_dev))
    model.free(gone)
    model.same(pool)
    remap, counts = ssd.pages_compact(pool)
    assert (remap.tolist(), counts.tolist()) == tuple(model.compact())
    ssd.device_status()
    model.same(pool)


def test_offsets_past_32_bits(ssd, cuda_dev):
    """A pool of 6 GiB in one array: the last pages start past 2^32 bytes."""
    n, per = 24, 64 << 20                                    # 24 pages of 256 MiB
    a = torch.empty(n, per, dtype=torch.float32, device=cuda_dev)
    a[:, 0], a[:, -1] = torch.arange(n, device=cuda_dev), torch.arange(n, device=cuda_dev) + 0.5
    a[22, 12345:12355] = 3.0
    pool = ssd.PagePool([a], 2, 2)
    ssd.pages_copy(pool, ints([22, 0], cuda_dev), ints([23, 21], cuda_dev))
    ssd.device_status()
    assert torch.equal(a[23], a[22]) and torch.equal(a[21], a[0])
    assert a[20, 0].item() == 20 and a[20, -1].item() == 20.5


def test_captured_and_replayed_on_another_stream(ssd, cuda_dev):
    pool, model = both(ssd, cuda_dev, 12, 6, 3)
    ssd.pages_append(pool, ints([0, 1], cuda_dev))
    saved = pool.meta.clone()
    parents, children, rows = ints([0, 1, 0], cuda_dev), ints([2, 3, 4], cuda_dev), ints([1, 2], cuda_dev)
    torch.cuda.synchronize()
    s = torch.cuda.Stream()

    def step():
        pool.meta.copy_(saved)
        ssd.pages_fork(pool, parents, children)
        ssd.pages_free(pool, rows)
        ssd.pages_append(pool, ints_rows, copy_last=True)
        return ssd.pages_compact(pool)

    ints_rows = ints([0, 5], cuda_dev)
    with torch.cuda.stream(s):
        step()
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g, stream=s):
        remap, counts = step()
    for _ in range(2):
        with torch.cuda.stream(s):
            g.replay()
        torch.cuda.synchronize()
        ssd.device_status()
        m = Model(make(cuda_dev, 12), 6, 3)
        assert m.append([0, 1], False) and m.fork([0, 1, 0], [2, 3, 4])
        m.free([1, 2])
        assert m.append([0, 5], True)
        assert (remap.tolist(), counts.tolist()) == tuple(m.compact())
        assert pool.refcount.tolist() == m.refs and pool.length.tolist() == [len(x) for x in m.rows]


def test_refusals_of_the_binding(ssd, cuda_dev):
    t = torch.zeros(4, 8, device=cuda_dev)
    for arrays, rows, mp in (([], 2, 2), ([t, t[:3]], 2, 2), ([t.t()], 2, 2), ([t.cpu()], 2, 2), ([t], 0, 2), ([t], 2, 0)):
        with pytest.raises(ValueError):
            ssd.PagePool(arrays, rows, mp)
    with pytest.raises(ssd.SSDError, match="UNSUPPORTED"):
        ssd.PagePool([t] * 129, 2, 2)
    pool = ssd.PagePool([t], 2, 2)
    for bad, err in ((torch.zeros(1, dtype=torch.int64, device=cuda_dev), TypeError), (torch.zeros(1, dtype=torch.int32), ValueError),
                     (torch.zeros(5, dtype=torch.int32, device=cuda_dev), ValueError)):
        with pytest.raises(err):
            ssd.pages_append(pool, bad)
    with pytest.raises(ValueError):
        ssd.pages_fork(pool, ints([0], cuda_dev), ints([0, 1], cuda_dev))


# --------------------------------------------------------------------------------- together
def test_sequences_branch_finish_and_move(ssd, cuda_dev):
    """Prompts into pages, a snapshot, parallel samples, finished rows, a compaction, tokens on
    what is left: every row's outputs equal the recurrence over its own tokens."""
    from oracle import linattn_oracle as LO
    H, Hk, K, V, rows = 4, 2, 64, 64, 8
    g = torch.Generator().manual_seed(7)
    draw = lambda n: (torch.randn(n, H, K, generator=g).bfloat16().to(cuda_dev), (torch.randn(n, Hk, K, generator=g) / 8).bfloat16().to(cuda_dev),  # noqa: E731
                      torch.randn(n, Hk, V, generator=g).bfloat16().to(cuda_dev))
    ld = torch.tensor([-0.01, -0.3], device=cuda_dev)
    layers = torch.randn(2, 16, Hk, V, K, device=cuda_dev)                   # two layers, both with the same inputs here
    pool = ssd.PagePool(list(layers), rows, 3)
    seen = {r: [] for r in range(rows)}                                      # each row's own tokens
    lens = [150, 40, 9]
    cu = ints([0, 150, 190, 199], cuda_dev)
    ssd.pages_append(pool, ints([0, 1, 2], cuda_dev))
    q, k, v = draw(199)
    for layer in layers:
        o, _ = ssd.linear_attn_fwd(q, k, v, ld, cu_seqlens=cu, final_state=layer, final_pages=pool.live[:3])
    for r, (a, n) in enumerate(zip((0, 150, 190), lens)):
        seen[r].append((q[a:a + n], k[a:a + n], v[a:a + n], o[a:a + n]))

    def step():
        qt, kt, vt = draw(rows)
        out = torch.zeros(rows, H, V, dtype=torch.bfloat16, device=cuda_dev)
        for layer in layers:
            ssd.linear_attn_update(layer, qt, kt, vt, ld, pages=pool.live, o=out)
        for r in range(rows):
            if int(pool.live[r]) >= 0:
                seen[r].append((qt[r:r + 1], kt[r:r + 1], vt[r:r + 1], out[r:r + 1]))
            else:
                assert not bool(out[r].any())

    step()
    ssd.pages_append(pool, ints([0, 2], cuda_dev), copy_last=True)           # snapshots of rows 0 and 2
    snapshot = layers[:, int(pool.table[0, 0])].clone()
    step()
    ssd.pages_fork(pool, ints([0, 0, 2, -1], cuda_dev), ints([3, 4, 5, 6], cuda_dev))
    seen[3], seen[4], seen[5] = list(seen[0]), list(seen[0]), list(seen[2])
    step()
    ssd.pages_free(pool, ints([0, 2, 1], cuda_dev))
    seen[0], seen[1], seen[2] = [], [], []
    _, counts = ssd.pages_compact(pool)
    step()
    ssd.device_status()
    # rows 3 and 4 share the snapshot of row 0, row 5 has one of row 2: 2 + 3 live pages
    assert counts.tolist()[0] == 5 and int(pool.refcount.max()) == 2
    assert torch.equal(layers[:, int(pool.table[3, 0])], snapshot) and pool.table[3, 0] == pool.table[4, 0]
    for r in (3, 4, 5):
        q, k, v, o = (torch.cat(x) for x in zip(*seen[r]))
        ref = LO.linattn(q, k, v, ld, K ** -0.5)
        # a prompt's bound (its scores and result are rounded to bf16), plus fp32 sums
        tol = 2.0 ** -8 * (ref["o"].abs() + ref["o_score"]) + 2.0 ** -14 * ref["o_mag"]
        assert bool(((o.double() - ref["o"]).abs() <= tol).all())
        page = int(pool.live[r])
        for layer in layers:
            assert bool(((layer[page].double() - ref["final"][0]).abs() <= 400 * 2.0 ** -23 * ref["s_mag"][0]).all())
    assert not torch.equal(layers[0, int(pool.live[3])], layers[0, int(pool.live[4])])


def test_copies_onto_themselves(ssd, cuda_dev):
    """Page x onto page x moves nothing and counts as a destination: x is no other pair's source
    or destination."""
    pool, model = both(ssd, cuda_dev, 8, 6, 2)
    ssd.pages_copy(pool, ints([3, 0, 5], cuda_dev), ints([3, 1, 5], cuda_dev))
    ssd.device_status()
    model.copy([3, 0, 5], [3, 1, 5])
    model.same(pool)
    for src, dst in (([3, 0], [3, 3]), ([0, 3], [3, 3]), ([3, 3], [3, 0]), ([3, 3], [3, 3])):
        ssd.pages_copy(pool, ints(src, cuda_dev), ints(dst, cuda_dev))
        with pytest.raises(ssd.SSDError, match="INVALID_ARG"):
            ssd.device_status()
        model.same(pool)


def test_threads_with_pools_of_other_sizes(ssd, cuda_dev):
    """Calls of host threads on pools whose requests take different amounts of shared memory (one
    bit a page: 56 and 128 KiB)."""
    from test_linattn_gpu import at_once
    jobs, arrays, keep = [], [], []
    for n in (458752, 1 << 20):
        a = torch.arange(n, dtype=torch.int32, device=cuda_dev).view(n, 1)
        pool, st = ssd.PagePool([a], 2, 2), torch.cuda.Stream()
        src, dst = ints([n - 1], cuda_dev), ints([0], cuda_dev)
        jobs.append((ssd._lib.ssd_pages_copy, (pool._ref, src.data_ptr(), dst.data_ptr(), 1, st.cuda_stream)))
        arrays.append(a)
        keep.append((pool, st, src, dst))
    torch.cuda.synchronize()
    assert at_once(jobs, 5000) == [0, 0]
    ssd.device_status()
    for a in arrays:
        assert int(a[0]) == len(a) - 1 and int(a[1]) == 1


def test_a_pool_dropped_while_another_stream_uses_it(ssd, cuda_dev):
    """Its workspace, metadata and arrays are not handed out again before that stream is done."""
    n = 1 << 20
    pool = ssd.PagePool([torch.zeros(n, 5, device=cuda_dev)], 2, 2)
    src, dst = ints([n - 1], cuda_dev), ints([0], cuda_dev)
    sizes = {t.data_ptr(): t.numel() * t.element_size() for t in (pool.workspace, pool.meta, pool.arrays[0])}
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    with torch.cuda.stream(side):
        torch.cuda._sleep(2_000_000_000)                   # about a second
        ssd.pages_copy(pool, src, dst)
        done = torch.cuda.Event()
        done.record()
    del pool
    fresh = [torch.empty(b, dtype=torch.uint8, device=cuda_dev) for b in sizes.values() for _ in range(2)]
    assert not done.query()
    assert not any(p <= t.data_ptr() < p + b for t in fresh for p, b in sizes.items())
    torch.cuda.synchronize()
    ssd.device_status()
