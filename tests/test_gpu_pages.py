"""PagePool (assign, grow, compact) against a plain model on the host, bit for bit, and a run
of the page calls with the stores and attentions that use the pages."""
import numpy as np
import pytest

torch = pytest.importorskip("torch")
if not torch.cuda.is_available():
    pytest.skip("needs a CUDA GPU", allow_module_level=True)

import serving_mog_decode_gb300 as mog
from serving_mog_decode_gb300 import buildlib

pytestmark = pytest.mark.gpu
DEV = torch.device("cuda:0")
D = 128


@pytest.fixture(scope="module", autouse=True)
def _built():
    buildlib.build()
    mog.lib()


def ints(x):
    return torch.tensor(x, dtype=torch.int32, device=DEV)


class Model:
    """The calls' definition, one sequence after another."""

    def __init__(self, n_pages, R, batch, pps):
        self.R, self.pps = R, pps
        self.table = [[] for _ in range(batch)]
        self.lengths = [0] * batch
        self.refs = np.zeros(n_pages, np.int64)
        self.content = np.arange(n_pages)  # which original page's bytes a page holds

    def assign(self, src):
        old, lens = [list(r) for r in self.table], list(self.lengths)
        for b, s in enumerate(src):
            if s == b or not -1 <= s < len(src):
                continue
            new = old[s] if s >= 0 else []
            for p in old[b]:
                self.refs[p] -= 1
            for p in new:
                self.refs[p] += 1
            self.table[b], self.lengths[b] = list(new), lens[s] if s >= 0 else 0

    def grow(self, n_new):
        keep = [list(r) for r in self.table], list(self.lengths), self.refs.copy(), self.content.copy()
        pos = list(self.lengths)
        free = [p for p in range(len(self.refs)) if self.refs[p] == 0]
        copies = []
        ok = all(n >= 0 and l + n <= self.pps * self.R for n, l in zip(n_new, self.lengths))
        for b, n in enumerate(n_new):
            if not ok or n == 0:
                continue
            row, ln = self.table[b], self.lengths[b]
            if ln % self.R and self.refs[row[-1]] > 1:
                if not free:
                    ok = False
                    break
                self.refs[row[-1]] -= 1
                copies.append((row[-1], free[0]))
                row[-1] = free.pop(0)
                self.refs[row[-1]] = 1
            while len(row) * self.R < ln + n:
                if not free:
                    ok = False
                    break
                row.append(free.pop(0))
                self.refs[row[-1]] = 1
            self.lengths[b] = ln + n
        if not ok:
            self.table, self.lengths, self.refs, self.content = keep
            return pos, [0] * len(n_new), False
        for s, d in copies:
            self.content[d] = self.content[s]
        return pos, list(n_new), True

    def compact(self):
        live = [p for p in range(len(self.refs)) if self.refs[p]]
        n = len(live)
        holes = [p for p in range(n) if not self.refs[p]]
        to = dict(zip([p for p in live if p >= n], holes))
        for s, d in to.items():
            self.refs[d], self.refs[s] = self.refs[s], 0
            self.content[d] = self.content[s]
        self.table = [[to.get(p, p) for p in r] for r in self.table]


def make(n_pages, R, batch, pps, H=2, layers=1, e4m3=False, seed=0, interleaved=False):
    g = torch.Generator(device=DEV).manual_seed(seed)

    def pool(*tail, dtype):
        if interleaved:  # pages of all pools side by side: a stride wider than a page
            return torch.randn((n_pages, 2) + tail, generator=g, device=DEV).to(dtype)[:, 1]
        return torch.randn((n_pages,) + tail, generator=g, device=DEV).to(dtype)

    dt = torch.float8_e4m3fn if e4m3 else torch.bfloat16
    K, V = ([pool(H, R, D, dtype=dt) for _ in range(layers)] for _ in range(2))
    kw = {}
    if e4m3:
        kw = dict(k_scale=[pool(H, R, dtype=torch.float32) for _ in range(layers)],
                  v_scale=[pool(H, R, dtype=torch.float32) for _ in range(layers)])
    return mog.PagePool(K, V, batch, pps, **kw)


def bits(t):
    return t.contiguous().view(torch.uint8).clone()


def tensors(pool):
    return pool.K + pool.V + (pool.k_scale or []) + (pool.v_scale or [])


def same(pool, model, before):
    want = np.full((pool.batch, model.pps), -1)
    for b, r in enumerate(model.table):
        want[b, :len(r)] = r
    assert np.array_equal(pool.block_table.cpu().numpy(), want)
    assert pool.lengths.tolist() == model.lengths
    assert np.array_equal(pool.refs.cpu().numpy(), model.refs)
    if before is not None:
        at = torch.from_numpy(model.content).to(DEV)
        for t, x in zip(tensors(pool), before):
            assert torch.equal(bits(t), x[at])


@pytest.mark.parametrize("n_pages,R,batch,pps,kw", [  # (the first two grow in one launch)
    (40, 16, 4, 12, {}), (60, 16, 7, 12, dict(H=1, e4m3=True, layers=2)), (300, 16, 9, 40, dict(layers=2, e4m3=True)), (97, 32, 33, 7, dict(interleaved=True)),
    (5000, 64, 70, 130, dict(H=1)), (17, 128, 1, 20, {}), (20011, 16, 1100, 33, dict(H=1, e4m3=True))])
def test_random_runs(n_pages, R, batch, pps, kw):
    """Random forks, frees, growth (until there is no room, too) and moves."""
    rng = np.random.default_rng(n_pages)
    pool, model = make(n_pages, R, batch, pps, **kw), Model(n_pages, R, batch, pps)
    before = [bits(t) for t in tensors(pool)]
    fails = 0
    for step in range(40):
        what = rng.integers(0, 10)
        if what < 4:
            src = np.where(rng.random(batch) < 0.6, np.arange(batch), rng.integers(-1, batch, batch))
            pool.assign(ints(src.tolist()))
            model.assign(src.tolist())
        elif what < 9:
            top = rng.choice([1, 2, R, 3 * R])
            n = np.where(rng.random(batch) < 0.5, rng.integers(0, top + 1, batch), 0)
            pos, granted = pool.grow(ints(n.tolist()))
            mp, mg, ok = model.grow(n.tolist())
            assert pos.tolist() == mp and granted.tolist() == mg
            assert pool.status() == (0 if ok else 8)
            fails += not ok
        else:
            pool.compact()
            model.compact()
        same(pool, model, before)
    assert pool.status() == 0
    print(f"{fails} of 40 steps found no room")


def test_grow_without_room_changes_nothing_and_recovers():
    pool, model = make(4, 16, 3, 4), Model(4, 16, 3, 4)
    for n in ([20, 16, 0], [0, 1, 20], [13, 0, 0], [0, 0, 65], [0, 0, 16]):
        got = pool.grow(ints(n))
        want = model.grow(n)
        assert got[0].tolist() == want[0] and got[1].tolist() == want[1]
        assert pool.status() == (0 if want[2] else 8)
        same(pool, model, None)
    pool.assign(ints([-1, 1, 2]))
    model.assign([-1, 1, 2])
    assert pool.grow(ints([0, 2, 0]))[1].tolist() == model.grow([0, 2, 0])[1] == [0, 2, 0]
    assert pool.status() == 0
    same(pool, model, None)


def test_bad_indices_are_left_out_and_reported():
    pool, model = make(16, 16, 3, 4), Model(16, 16, 3, 4)
    pool.grow(ints([20, 5, 0]))
    model.grow([20, 5, 0])
    pool.assign(ints([7, -2, 0]))
    model.assign([7, -2, 0])
    same(pool, model, None)
    assert pool.status() == 5 and pool.status() == 0
    pos, granted = pool.grow(ints([1, -1, 1]))
    assert granted.tolist() == [0, 0, 0] and pool.status() == 5
    same(pool, model, None)
    # a table that names pages outside the pool: the call refuses, nothing is read there
    keep = pool.block_table.clone()
    pool.block_table[1, 0] = 1 << 30
    assert pool.grow(ints([0, 1, 0]))[1].tolist() == [0, 0, 0] and pool.status() == 5
    pool.compact()
    pool.assign(ints([0, -1, 2]))
    assert pool.status() == 5
    pool.block_table.copy_(keep)


def test_sequences_exchange_pages():
    """Every sequence takes another's pages at once: all sources are read first."""
    pool, model = make(64, 16, 5, 8), Model(64, 16, 5, 8)
    pool.grow(ints([100, 3, 0, 40, 17]))
    model.grow([100, 3, 0, 40, 17])
    for src in ([1, 2, 3, 4, 0], [4, 4, 4, 4, 4], [0, 1, 2, -1, 0], [2, 2, 1, 1, 3]):
        pool.assign(ints(src))
        model.assign(src)
        same(pool, model, None)


def test_the_last_holder_keeps_a_shared_page():
    pool, model = make(16, 16, 3, 4), Model(16, 16, 3, 4)
    before = [bits(t) for t in tensors(pool)]
    for n, src in (([20, 0, 0], [0, 0, 0]), ([1, 1, 1], None)):
        pool.grow(ints(n))
        model.grow(n)
        if src:
            pool.assign(ints(src))
            model.assign(src)
        same(pool, model, before)
    assert len(set(pool.block_table[:, 1].tolist())) == 3 and pool.refs[pool.block_table[2, 1]].item() == 1


def test_more_pools_than_one_copy_launch_holds():
    pool, model = make(12, 16, 2, 4, H=1, layers=40), Model(12, 16, 2, 4)
    before = [bits(t) for t in tensors(pool)]
    pool.grow(ints([20, 0]))
    model.grow([20, 0])
    pool.assign(ints([0, 0]))
    model.assign([0, 0])
    pool.grow(ints([1, 1]))
    model.grow([1, 1])
    same(pool, model, before)
    pool.assign(ints([-1, 1]))
    model.assign([-1, 1])
    pool.compact()
    model.compact()
    same(pool, model, before)


@pytest.mark.parametrize("kw", [{}, dict(R=64, H=8)])  # growth in one launch, in two
def test_page_calls_in_a_graph(kw):
    pool = make(64, kw.get("R", 16), 4, 8, H=kw.get("H", 2))
    n, src = ints([30, 0, 0, 0]), ints([0, 0, 0, -1])
    pool.grow(n)
    one = ints([0, 1, 1, 1])
    pool.assign(src)
    pool.grow(one)
    torch.cuda.synchronize()
    want = pool.block_table.clone(), pool.refs.clone(), pool.lengths.clone()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        pool.assign(src)
        pos, granted = pool.grow(one)
    for _ in range(3):  # each replay gives the samples back and forks them again
        graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip((pool.block_table, pool.refs, pool.lengths), want))
        assert pos.tolist() == [30, 30, 30, 0] and granted.tolist() == [0, 1, 1, 1]


def test_compaction_in_a_graph():
    pool, model = make(64, 16, 4, 8), Model(64, 16, 4, 8)
    before = [bits(t) for t in tensors(pool)]
    src, n = ints([2, 3, -1, -1]), ints([0, 0, 70, 33])
    for m, x in ((pool, ints([70, 33, 70, 33])), (model, [70, 33, 70, 33])):
        m.grow(x)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        pool.assign(src)
        pool.compact()
        pool.grow(n)
    for _ in range(4):
        graph.replay()
        model.assign(src.tolist())
        model.compact()
        model.grow(n.tolist())
        same(pool, model, before)


def test_pool_refusals():
    K = torch.zeros((8, 2, 16, D), dtype=torch.bfloat16, device=DEV)
    for bad in (K[:, :, :, :64], K.transpose(1, 2), K[:4]):
        with pytest.raises(ValueError):
            mog.PagePool(K, bad, 2, 4)
    with pytest.raises(ValueError):
        mog.PagePool([K, K], [K], 2, 4)
    with pytest.raises(ValueError):  # e4m3 rows without scales, scales with bf16 rows
        mog.PagePool(K.to(torch.float8_e4m3fn), K.to(torch.float8_e4m3fn), 2, 4)
    with pytest.raises(ValueError):
        mog.PagePool(K, K.clone(), 2, 4, k_scale=K[..., 0].float(), v_scale=K[..., 0].float())
    with pytest.raises(ValueError):
        mog.PagePool(K, K.clone(), 2, 4, lengths=torch.zeros(3, dtype=torch.int32, device=DEV))
    with pytest.raises(mog.MogError, match="SHAPE"):
        mog.PagePool(K, K.clone(), 5000, 4)
    pool = mog.PagePool(K, K.clone(), 2, 4)
    with pytest.raises(ValueError):
        pool.assign(torch.zeros(3, dtype=torch.int32, device=DEV))
    with pytest.raises(ValueError):
        pool.grow(torch.zeros(2, dtype=torch.int64, device=DEV))


def pow2(e):
    return ((e.long() + 1023) << 52).view(torch.float64)


def nearest_rows(x):
    """Stored value of bf16 rows: e4m3 with the least power-of-two scale (64 bits)."""
    x = x.double()
    amax = x.abs().amax(-1, keepdim=True)
    sc = pow2(torch.floor(torch.log2(amax / 448)) - 1)
    for _ in range(2):
        sc = torch.where(448 * sc < amax, 2 * sc, sc)
    m, e = torch.frexp(x / sc)
    step = pow2((e - 1).clamp_min(-6) - 3)
    return torch.round(x / sc / step) * step * sc


@pytest.mark.parametrize("e4m3", [True, False])
def test_serving_run(e4m3):
    """Prompts in, samples forked, tokens appended and attended each step, sequences that end
    and pages that move: the attentions see each sequence's own rows throughout."""
    H, G, R, batch, pps, layers = 2, 4, 16, 7, 24, 2
    g = torch.Generator(device=DEV).manual_seed(5)
    pool = make(90, R, batch, pps, H=H, layers=layers, e4m3=e4m3)
    rows = [[[torch.zeros((0, H, D), dtype=torch.float64, device=DEV) for _ in range(2)] for _ in range(batch)]
            for _ in range(layers)]
    lam = 0.2 * torch.randn((4, 64), generator=g, device=DEV)

    def append(n_new):
        pos, granted = pool.grow(ints(n_new))
        T = max(n_new)
        for l in range(layers):
            new = [torch.randn((batch, T, H, D), generator=g, device=DEV).bfloat16() for _ in range(2)]
            mog.kv_store(pool.cache(l), None, pos, granted, *new)
            for b, n in enumerate(n_new):
                for i in range(2):
                    x = new[i][b, :n]
                    rows[l][b][i] = torch.cat([rows[l][b][i], nearest_rows(x) if e4m3 else x.double()])

    def assign(src):
        pool.assign(ints(src))
        for l in range(layers):
            old = list(rows[l])
            rows[l][:] = [[x.clone() for x in old[s]] if s >= 0 else [x[:0] for x in old[b]] for b, s in enumerate(src)]

    def attend():
        q = torch.randn((batch, H * G, D), generator=g, device=DEV).bfloat16()
        outs = []
        for l in range(layers):
            c = pool.cache(l)
            dense = mog.dense_decode(c, None, pool.lengths, pps * R, q)
            diff = mog.diff_decode(c, None, pool.lengths, pps * R, q, lam, 0.5)
            w = torch.exp((lam[0] * lam[1]).sum().double()) - torch.exp((lam[2] * lam[3]).sum().double()) + 0.5
            for b in range(batch):
                K, V = rows[l][b]
                for h in range(H * G):
                    if K.shape[0] == 0:
                        assert (dense[b, h] == 0).all() and (diff[b, h] == 0).all()
                        continue
                    k, v, x = K[:, h // G], V[:, h // G], q[b, h].double()
                    ref = torch.softmax(k @ x / D ** 0.5, 0) @ v
                    a = (torch.softmax(k[:, :64] @ x[:64] / 8, 0) - w * torch.softmax(k[:, 64:] @ x[64:] / 8, 0)) @ v
                    dref = 0.5 * a / torch.sqrt((a * a).mean() + 1e-5)
                    # weights within 2^-15 of their own size: fp32 logits of |s| < 40 and their exponentials
                    tol = 2.0 ** -14
                    assert (dense[b, h] - ref).norm() <= tol * v.abs().max() * D ** 0.5
                    assert (diff[b, h] - dref).norm() <= 8 * tol * v.abs().max() * D ** 0.5 / max((a * a).mean().sqrt(), 1e-3)
            outs += [dense, diff]
        return q, outs

    append([100, 37, 16, 0, 0, 0, 0])
    attend()
    assign([0, 1, 2, 0, 0, 1, 2])        # samples of the prompts
    for _ in range(3):
        append([0, 1, 1, 1, 1, 1, 1])
        attend()
    assign([-1, 4, 2, 3, 4, 3, 6])       # one prompt ends, samples take each other's place
    append([50, 1, 0, 17, 1, 1, 33])
    q, outs = attend()
    pool.compact()
    for l in range(layers):              # the same rows in other pages: the same bits
        c = pool.cache(l)
        assert torch.equal(mog.dense_decode(c, None, pool.lengths, pps * R, q), outs[2 * l])
        assert torch.equal(mog.diff_decode(c, None, pool.lengths, pps * R, q, lam, 0.5), outs[2 * l + 1])
    live = int((pool.refs > 0).sum())
    assert int(pool.refs[live:].abs().sum()) == 0 and pool.status() == 0
    append([1] * batch)
    attend()


def test_no_page_outside_the_plan_is_written():
    """Pools and tables inside larger buffers: what is around them stays."""
    g = torch.Generator(device=DEV).manual_seed(9)
    big = [torch.randn((20, 2, 16, D), generator=g, device=DEV).bfloat16() for _ in range(2)]
    keep = [b.clone() for b in big]
    table = torch.full((6, 4), 77, dtype=torch.int32, device=DEV)
    table[1:5] = -1
    pool = mog.PagePool(big[0][2:-2], big[1][2:-2], 4, 4, block_table=table[1:5])
    model = Model(16, 16, 4, 4)
    for n, src in (([20, 0, 16, 3], [0, 0, 0, 3]), ([1, 1, 1, 1], [-1, 1, 2, 3]), ([0, 0, 0, 5], [1, 2, 3, 1])):
        pool.grow(ints(n))
        model.grow(n)
        pool.assign(ints(src))
        model.assign(src)
        pool.compact()
        model.compact()
        same(pool, model, None)
    assert (table[0] == 77).all() and (table[5] == 77).all()
    at = torch.from_numpy(model.content).to(DEV)
    for b, k in zip(big, keep):
        assert torch.equal(b[:2], k[:2]) and torch.equal(b[-2:], k[-2:]) and torch.equal(b[2:-2], k[2:-2][at])


def test_many_holders_of_one_last_page():
    """4096 sequences that share a partly filled page all grow: all but the last copy it."""
    B = 4096
    pool, model = make(B + 8, 16, B, 2, H=1), Model(B + 8, 16, B, 2)
    first = [5] + [0] * (B - 1)
    pool.grow(ints(first))
    model.grow(first)
    pool.assign(ints([0] * B))
    model.assign([0] * B)
    before = [bits(t) for t in tensors(pool)]
    model.content = np.arange(B + 8)
    pool.grow(ints([1] * B))
    model.grow([1] * B)
    same(pool, model, before)
    assert pool.status() == 0
