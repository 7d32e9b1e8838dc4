"""Measured cases of the paged, shared and 8-bit KV cache and of the decode attentions that
read it: inputs, the plain form of each operator in elementary torch operations, and the
calls of this package (`own`).

  store    new keys and values rounded to e4m3 with a scale per row, into a cache's pages
  dense8   full-scan decode attention over an e4m3 cache, one new token per sequence
  diff     differential decode attention (the difference of two softmax maps, normalised)
  fork     the samples of a prompt take its pages, then grow by tokens of their own: the
           partly filled last page becomes private
  compact  half of the sequences finish, the pages that live move to the front of the pool,
           new sequences take the pages behind them
"""
import math

import torch

own = False

D = 128          # row of a cache; a differential head is two halves of D/2
E4M3_MAX = 448.0


# ------------------------------------------------------------------------------- the cases

def listed():
    return [
        # a decode step's new token of each sequence of a batch: latency
        dict(name="store-step", op="store", B=8, H=8, T=1, n=4096, page=64, ragged=False),
        # prompts of different lengths written into pages behind what is there
        dict(name="store-prompt", op="store", B=4, H=8, T=8191, n=4096, page=16, ragged=True),
        # a short chat in small pages: latency
        dict(name="dense8-1000", op="dense8", B=1, H=8, G=4, n=1000, page=16, ragged=False, out="f32"),
        # a batch of sequences between 16K and 64K with a KV head per query head
        dict(name="dense8-varlen", op="dense8", B=8, H=32, G=1, n=65536, page=64, ragged=True, out="bf16"),
        # one sequence of 1M tokens in a contiguous cache
        dict(name="dense8-1m", op="dense8", B=1, H=8, G=4, n=1048576, page=0, ragged=False, out="f32"),
        # two short sequences in pages: latency
        dict(name="diff-4k", op="diff", B=2, H=8, G=4, n=4096, page=64, ragged=True, cache="bf16", out="f32"),
        # one sequence of 32K tokens in a contiguous bf16 cache
        dict(name="diff-32k", op="diff", B=1, H=8, G=4, n=32768, page=0, ragged=False, cache="bf16", out="bf16"),
        # a batch at 128K with five heads on each KV head, in 8-bit pages
        dict(name="diff-128k", op="diff", B=4, H=8, G=5, n=131072, page=64, ragged=False, cache="e4m3", out="f32"),
        # four samples of each of two prompts
        dict(name="fork-8", op="fork", P=2, S=4, H=8, page=16, n=1000, T=1, layers=1),
        # eight samples of each of 32 prompts, pages of two layers
        dict(name="fork-256", op="fork", P=32, S=8, H=8, page=64, n=8192, T=1, layers=2),
        # four short sequences of which two finish
        dict(name="compact-4", op="compact", B=4, H=8, page=16, n=1000, layers=1),
        # 16 sequences of up to 16K tokens
        dict(name="compact-16", op="compact", B=16, H=8, page=64, n=16384, layers=1),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["store", "dense8", "diff", "fork", "compact"])
    page = rng.choice([16, 32, 64, 128])
    if op == "store":
        H = rng.choice([1, 2, 4, 8, 32])
        B = _log(rng, 1, 64)
        T = _log(rng, 1, max(1, min(8191, 262144 // (B * H))))
        return dict(op=op, B=B, H=H, T=T, n=_log(rng, 1, 4096), page=page, ragged=rng.random() < 0.5)
    if op in ("dense8", "diff"):
        H = rng.choice([1, 2, 4, 8, 32])
        G = rng.choice([1, 2, 3, 4, 5, 8] if op == "diff" else [1, 2, 3, 4, 5, 7, 8, 12, 16])
        B = _log(rng, 1, 16)
        n = _log(rng, 1, min(1 << 20, (1 << 22) // (B * H)))
        case = dict(op=op, B=B, H=H, G=G, n=n, page=rng.choice([0, page]), ragged=rng.random() < 0.5,
                    out=rng.choice(["f32", "bf16"]))
        if op == "diff":
            case["cache"] = rng.choice(["bf16", "e4m3"])
        return case
    layers = rng.choice([1, 2])
    if op == "fork":
        P, S = _log(rng, 1, 32), _log(rng, 1, 8)
        n = _log(rng, 1, min(8192, 262144 // P))
        return dict(op=op, P=P, S=S, H=rng.choice([1, 2, 8]), page=page, n=n, T=_log(rng, 1, 64), layers=layers)
    B = 2 * _log(rng, 1, 16)
    n = _log(rng, 1, min(32768, 131072 // B))
    return dict(op=op, B=B, H=rng.choice([1, 2, 8]), page=page, n=n, layers=layers)


# ------------------------------------------------------------------------------ the inputs

def _ceil(a, b):
    return -(-a // b)


def _lengths(case, gen, lo, hi, count):
    """int32 lengths on the device: hi each, or spread over [lo, hi] when the batch is ragged."""
    if not case.get("ragged", True):
        return torch.full((count,), hi, dtype=torch.int32, device="cuda")
    return torch.randint(lo, hi + 1, (count,), generator=gen, device="cuda", dtype=torch.int32)


def _keys(gen, slabs, H, rows):
    """bf16 [slabs, H, rows, D] keys around 64 centres of their head, as attention keys cluster."""
    centres = torch.randn((H, 64, D), generator=gen, device="cuda")
    z = torch.randint(0, 64, (slabs, H, rows), generator=gen, device="cuda")
    k = torch.randn((slabs, H, rows, D), generator=gen, device="cuda").mul_(0.5)
    k += centres[torch.arange(H, device="cuda")[None, :, None], z]
    return k.bfloat16(), centres


def _quantised(x):
    """(e4m3 codes, fp32 scale of each row) of bf16 rows: largest magnitude at 448."""
    scale = x.float().abs().amax(-1).clamp_min(1e-20) / E4M3_MAX
    return (x.float() / scale[..., None]).to(torch.float8_e4m3fn), scale


def _prepare_store(case, gen):
    B, H, T, R = case["B"], case["H"], case["T"], case["page"]
    pos = _lengths(case, gen, case["n"] // 2, case["n"], B)
    count = _lengths(case, gen, T // 2, T, B)
    pps = _ceil(case["n"] + T, R)
    table = torch.randperm(B * pps, generator=gen, device="cuda").int().view(B, pps)
    kv = torch.randn((B, T, 2 * H, D), generator=gen, device="cuda")  # one fused projection's output
    kv *= torch.exp(torch.randn((B, T, 2 * H, 1), generator=gen, device="cuda"))
    kv = kv.bfloat16()
    pool = [torch.zeros((B * pps, H, R, D), device="cuda").to(torch.float8_e4m3fn) for _ in range(2)]
    scales = [torch.ones((B * pps, H, R), device="cuda") for _ in range(2)]
    return dict(case=case, K=pool[0], V=pool[1], ks=scales[0], vs=scales[1], table=table, pos=pos, count=count,
                k_new=kv[:, :, :H], v_new=kv[:, :, H:])


def _prepare_decode(case, gen):
    B, H, G, n, R = case["B"], case["H"], case["G"], case["n"], case["page"]
    lengths = _lengths(case, gen, max(1, n // 4), n, B)
    if R:
        pps = _ceil(n, R)
        slabs, rows = B * pps, R
        table = torch.randperm(slabs, generator=gen, device="cuda").int().view(B, pps)
    else:
        slabs, rows, table = B, n, None
    K, centres = _keys(gen, slabs, H, rows)
    V = torch.randn((slabs, H, rows, D), generator=gen, device="cuda").bfloat16()
    pick = torch.randint(0, 64, (B, H, G), generator=gen, device="cuda")
    q = 0.5 * centres[torch.arange(H, device="cuda")[None, :, None], pick]
    q = (q + 0.5 * torch.randn((B, H, G, D), generator=gen, device="cuda")).view(B, H * G, D).bfloat16()
    s = dict(case=case, lengths=lengths, table=table, q=q, K=K, V=V)
    if case.get("cache", "e4m3") == "e4m3":
        s["K"], s["ks"] = _quantised(K)
        s["V"], s["vs"] = _quantised(V)
    if case["op"] == "diff":
        s["lam"] = 0.1 * torch.randn((4, D // 2), generator=gen, device="cuda")
        s["gamma"] = 1.0 + 0.1 * torch.randn((D,), generator=gen, device="cuda")
        s["lambda_init"], s["eps"] = 0.8 - 0.6 * math.exp(-0.3 * 4), 1e-5  # of the fifth layer
    return s


def _pools(gen, layers, n_pages, H, R):
    return [[torch.randn((n_pages, H, R, D), generator=gen, device="cuda", dtype=torch.bfloat16)
             for _ in range(layers)] for _ in range(2)]


def _tables(lengths, batch, pps, R, n_pages, gen):
    """A block table of `lengths` with pages in a random order (-1 past the end), and the
    number of holders of every page."""
    perm = torch.randperm(n_pages, generator=gen, device="cuda").int()
    used = (lengths.long() + R - 1) // R
    first = used.cumsum(0) - used
    slot = torch.arange(pps, device="cuda")
    at = (first[:, None] + slot).clamp_max(n_pages - 1)
    table = torch.where(slot < used[:, None], perm[at], -1).int()
    table = torch.cat([table, torch.full((batch - len(lengths), pps), -1, dtype=torch.int32, device="cuda")])
    refs = torch.zeros(n_pages + 1, dtype=torch.int32, device="cuda")
    refs.scatter_add_(0, torch.where(table < 0, n_pages, table).long().view(-1), torch.ones_like(table).view(-1))
    return table, refs[:n_pages].clone()


def _prepare_fork(case, gen):
    P, S, H, R, n, T = (case[k] for k in ("P", "S", "H", "page", "n", "T"))
    batch, pps = P * (1 + S), _ceil(n + T, R)
    n_pages = P * _ceil(n, R) + P * S * (_ceil(T, R) + 1)
    lengths = _lengths(case, gen, max(1, n // 2), n, P)
    table, refs = _tables(lengths, batch, pps, R, n_pages, gen)
    rows = torch.arange(batch, device="cuda")
    K, V = _pools(gen, case["layers"], n_pages, H, R)
    return dict(case=case, K=K, V=V, table=table, refs=refs, lengths=torch.cat([lengths, lengths.new_zeros(P * S)]),
                src=torch.where(rows < P, rows, (rows - P) // S).int(), grow=torch.where(rows < P, 0, T).int())


def _prepare_compact(case, gen):
    B, H, R, n = (case[k] for k in ("B", "H", "page", "n"))
    pps = _ceil(n, R)
    n_pages = B * pps
    lengths = _lengths(case, gen, max(1, n // 2), n, B)
    table, refs = _tables(lengths, B, pps, R, n_pages, gen)
    rows = torch.arange(B, device="cuda")
    K, V = _pools(gen, case["layers"], n_pages, H, R)
    half = B // 2
    return dict(case=case, K=K, V=V, table=table, refs=refs, lengths=lengths,
                src=torch.where(rows < half, rows + half, -1).int(), grow=torch.where(rows < half, 0, lengths).int())


def prepare(case, seed):
    gen = torch.Generator(device="cuda").manual_seed(seed)
    make = dict(store=_prepare_store, dense8=_prepare_decode, diff=_prepare_decode, fork=_prepare_fork,
                compact=_prepare_compact)
    return make[case["op"]](case, gen)


# -------------------------------------------------------------------------- the plain forms

def _store_rows(pool, scales, table, b, t, pos, x):
    """One of the two pools: rows x [m, H, D] (fp32) to position pos of sequence b."""
    R = pool.shape[2]
    amax = torch.where(torch.isfinite(x), x.abs(), 0.0).amax(-1)
    m, e = torch.frexp(amax)
    e = torch.where(m > 0.875, e - 8, e - 9).clamp_min(-126)  # the least e with amax <= 448 * 2^e
    scale = torch.where(amax > 0, ((e + 127) << 23).view(torch.float32), 1.0)
    code = (x / scale[..., None]).clamp(-E4M3_MAX, E4M3_MAX).to(torch.float8_e4m3fn)
    page, row = table[b, pos // R].long(), pos % R
    pool.view(torch.uint8)[page, :, row] = code.view(torch.uint8)
    scales[page, :, row] = scale


def _plain_store(s):
    T = s["k_new"].shape[1]
    b, t = torch.nonzero(torch.arange(T, device="cuda") < s["count"][:, None], as_tuple=True)
    pos = s["pos"].long()[b] + t
    _store_rows(s["K"], s["ks"], s["table"], b, t, pos, s["k_new"][b, t].float())
    _store_rows(s["V"], s["vs"], s["table"], b, t, pos, s["v_new"][b, t].float())
    return dict(K=s["K"], V=s["V"], ks=s["ks"], vs=s["vs"])


def _plain_rows(s, which, scale):
    """fp32 [B, H, n, D] rows of the cache in order."""
    x, table = s[which], s["table"]
    if table is not None:
        idx = table.long()
        x = (x.view(torch.uint8)[idx].view(x.dtype)).transpose(1, 2)  # [B, H, pages, R, D]
        x = x.flatten(2, 3)
    x = x.float()
    if scale in s:
        sc = s[scale]
        x *= (sc if table is None else sc[table.long()].transpose(1, 2).flatten(2, 3))[..., None]
    return x


def _plain_softmax_v(q, K, V, lengths, tau):
    """softmax(tau q K^T) V over each sequence's rows; zeros where there are none."""
    logit = torch.matmul(q, K.transpose(-1, -2)) * tau
    seen = torch.arange(K.shape[2], device="cuda") < lengths.view(-1, 1, 1, 1)
    logit = torch.where(seen, logit, float("-inf"))
    top = logit.amax(-1, keepdim=True)
    w = torch.where(seen, torch.exp(logit - top), 0.0)
    total = w.sum(-1, keepdim=True)
    return torch.matmul(w, V) / torch.where(total > 0, total, 1.0)


def _out_type(case):
    return torch.float32 if case["out"] == "f32" else torch.bfloat16


def _plain_dense8(s):
    B, H, G = (s["case"][k] for k in ("B", "H", "G"))
    K, V = _plain_rows(s, "K", "ks"), _plain_rows(s, "V", "vs")
    out = _plain_softmax_v(s["q"].float().view(B, H, G, D), K, V, s["lengths"], 1 / math.sqrt(D))
    return out.view(B, H * G, D).to(_out_type(s["case"]))


def _plain_diff(s):
    B, H, G = (s["case"][k] for k in ("B", "H", "G"))
    K, V = _plain_rows(s, "K", "ks"), _plain_rows(s, "V", "vs")
    q, h, tau = s["q"].float().view(B, H, G, D), D // 2, 1 / math.sqrt(D // 2)
    a1 = _plain_softmax_v(q[..., :h], K[..., :h], V, s["lengths"], tau)
    a2 = _plain_softmax_v(q[..., h:], K[..., h:], V, s["lengths"], tau)
    lam = s["lam"]
    weight = torch.exp((lam[0] * lam[1]).sum()) - torch.exp((lam[2] * lam[3]).sum()) + s["lambda_init"]
    a = a1 - weight * a2
    a = a * torch.rsqrt(a.square().mean(-1, keepdim=True) + s["eps"]) * s["gamma"] * (1 - s["lambda_init"])
    return a.view(B, H * G, D).to(_out_type(s["case"]))


def _plain_assign(s):
    """Sequence b becomes another holder of the pages that src[b] held before the call (-1: of none)."""
    src, table, n_pages = s["src"].long(), s["table"], s["refs"].shape[0]
    new = torch.where(src[:, None] >= 0, table[src.clamp_min(0)], -1)
    lengths = torch.where(src >= 0, s["lengths"][src.clamp_min(0)], 0)
    held = torch.zeros(n_pages + 1, dtype=torch.int32, device="cuda")
    one = torch.ones_like(table).view(-1)
    held.scatter_add_(0, torch.where(new < 0, n_pages, new).long().view(-1), one)
    held.scatter_add_(0, torch.where(table < 0, n_pages, table).long().view(-1), -one)
    s["refs"] += held[:n_pages]
    table.copy_(new)
    s["lengths"].copy_(lengths)


def _plain_grow(s):
    """Pages for n_new more tokens of every sequence, lowest free page first; a partly filled
    last page with other holders is copied first, as if the sequences came one after another."""
    grow, table, refs, lengths, R = s["grow"], s["table"], s["refs"], s["lengths"], s["K"][0].shape[2]
    B, pps = table.shape
    rows, slot = torch.arange(B, device="cuda"), torch.arange(pps, device="cuda")
    old = (lengths + R - 1) // R
    new = torch.where(grow > 0, (lengths + grow + R - 1) // R, old)
    tail = table[rows, (old - 1).clamp_min(0).long()]
    part = (grow > 0) & (lengths % R != 0)
    same = (tail[:, None] == tail[None]) & part[:, None] & part[None]
    before = (same & (rows[None] < rows[:, None])).sum(1)
    private = part & (refs[tail.clamp_min(0).long()] - before > 1)
    want = ((slot >= old[:, None]) & (slot < new[:, None])) | (private[:, None] & (slot == old[:, None] - 1))
    order = want.view(-1).int().cumsum(0).view(B, pps)
    page = torch.searchsorted((refs == 0).int().cumsum(0).int(), order.int()).int()
    moved = private.nonzero()[:, 0]
    src, dst = tail[moved].long(), page[moved, old[moved].long() - 1].long()
    for pool in s["K"] + s["V"]:
        pool[dst] = pool[src]
    refs.scatter_add_(0, src, torch.full_like(moved, -1, dtype=torch.int32))
    refs[page[want].long()] = 1
    table.copy_(torch.where(want, page, table))
    pos = lengths.clone()
    lengths += grow
    return pos


def _plain_compact(s):
    """The i-th live page behind the first n_live takes the i-th free place among them."""
    refs, table = s["refs"], s["table"]
    live = refs > 0
    front = torch.arange(refs.shape[0], device="cuda") < live.sum()
    dst, src = (~live & front).nonzero()[:, 0], (live & ~front).nonzero()[:, 0]
    for pool in s["K"] + s["V"]:
        pool[dst] = pool[src]
    at = torch.arange(refs.shape[0], device="cuda", dtype=torch.int32)
    at[src] = dst.int()
    table.copy_(torch.where(table >= 0, at[table.clamp_min(0).long()], -1))
    refs[dst] = refs[src]
    refs[src] = 0


def _pages_out(s, pos):
    return dict(table=s["table"], refs=s["refs"], lengths=s["lengths"], pos=pos,
                K=[x.view(torch.int16) for x in s["K"]], V=[x.view(torch.int16) for x in s["V"]])


def _plain_fork(s):
    _plain_assign(s)
    return _pages_out(s, _plain_grow(s))


def _plain_compact_pass(s):
    _plain_assign(s)
    _plain_compact(s)
    return _pages_out(s, _plain_grow(s))


# --------------------------------------------------------------------- this package's calls

def _own_cache(s):
    """The cache object that a program makes once, when it lays its cache out."""
    if "cache" not in s:
        import serving_mog_decode_gb300 as mog
        if s["table"] is None:
            s["cache"] = mog.KV8(s["K"], s["V"], s["ks"], s["vs"]) if "ks" in s else s["K"]
        elif "ks" in s:
            s["cache"] = mog.PagedKV8(s["K"], s["V"], s["ks"], s["vs"], s["table"], s["K"].shape[2])
        else:
            s["cache"] = mog.PagedKV(s["K"], s["V"], s["table"], s["K"].shape[2])
    return s["cache"], (s["V"] if s["cache"] is s["K"] else None)


def _own_pool(s):
    if "pool" not in s:
        import serving_mog_decode_gb300 as mog
        s["pool"] = mog.PagePool(s["K"], s["V"], *s["table"].shape, block_table=s["table"], lengths=s["lengths"],
                                 refs=s["refs"])
    return s["pool"]


def _own_store(s):
    import serving_mog_decode_gb300 as mog
    K, V = _own_cache(s)
    mog.kv_store(K, V, s["pos"], s["count"], s["k_new"], s["v_new"])
    return dict(K=s["K"], V=s["V"], ks=s["ks"], vs=s["vs"])


def _own_out(s):
    return torch.empty(s["q"].shape, dtype=_out_type(s["case"]), device="cuda")


def _own_dense8(s):
    import serving_mog_decode_gb300 as mog
    K, V = _own_cache(s)
    return mog.dense_decode(K, V, s["lengths"], s["case"]["n"], s["q"], out=_own_out(s))


def _own_diff(s):
    import serving_mog_decode_gb300 as mog
    K, V = _own_cache(s)
    return mog.diff_decode(K, V, s["lengths"], s["case"]["n"], s["q"], s["lam"], s["lambda_init"], gamma=s["gamma"],
                           eps=s["eps"], out=_own_out(s))


def _own_fork(s):
    pool = _own_pool(s)
    pool.assign(s["src"])
    pos, _ = pool.grow(s["grow"])
    return _pages_out(s, pos)


def _own_compact_pass(s):
    pool = _own_pool(s)
    pool.assign(s["src"])
    pool.compact()
    pos, _ = pool.grow(s["grow"])
    return _pages_out(s, pos)


def run(state):
    op = state["case"]["op"]
    if own:
        return dict(store=_own_store, dense8=_own_dense8, diff=_own_diff, fork=_own_fork,
                    compact=_own_compact_pass)[op](state)
    return dict(store=_plain_store, dense8=_plain_dense8, diff=_plain_diff, fork=_plain_fork,
                compact=_plain_compact_pass)[op](state)


# ------------------------------------------------------------------------ what a pass needs

def work(case):
    """Expected bytes and operations over the distribution of ragged lengths."""
    op = case["op"]
    if op == "store":
        rows = case["B"] * case["H"] * (0.75 if case["ragged"] and case["T"] > 1 else 1) * case["T"]
        return dict(bytes=2 * rows * (2 * D + D + 4), flops=2 * rows * 3 * D)
    if op in ("dense8", "diff"):
        B, H, G = case["B"], case["H"], case["G"]
        rows = B * H * case["n"] * (0.625 if case["ragged"] else 1)
        row_bytes = D + 4 if case.get("cache", "e4m3") == "e4m3" else 2 * D
        maps = 3 * D if op == "diff" else 2 * D  # a differential head: D for both logits, D for each map's values
        out = 4 if case["out"] == "f32" else 2
        return dict(bytes=2 * rows * row_bytes + B * H * G * D * (2 + out), flops=2 * rows * G * maps)
    page = 2 * case["layers"] * case["H"] * case["page"] * D * 2
    if op == "fork":
        seqs, used = case["P"] * (1 + case["S"]), _ceil(0.75 * case["n"], case["page"])
        moved = case["P"] * case["S"]
        table = 8 * used * seqs
    else:
        seqs, used = case["B"], _ceil(0.75 * case["n"], case["page"])
        moved = (seqs // 2) * used
        table = 8 * used * seqs
    return dict(bytes=2 * moved * page + table, flops=0)


# ---------------------------------------------------- the definitions, in 64 bits, row by row

def _e4m3_nearest(y):
    """The nearest e4m3 value of float64 y, ties to the even mantissa, saturating."""
    step = torch.exp2(torch.floor(torch.log2(y.abs().clamp_min(2.0 ** -6))) - 3)
    return (torch.round(y / step) * step).clamp(-E4M3_MAX, E4M3_MAX)


def _exact_store(case, seed):
    s = prepare(case, seed)
    R, T = case["page"], case["T"]
    out = {}
    for pool, scales, new in (("K", "ks", "k_new"), ("V", "vs", "v_new")):
        values, scale = s[pool].double(), s[scales].double()
        for b in range(case["B"]):
            count, pos = int(s["count"][b]), int(s["pos"][b])
            at = torch.arange(pos, pos + count, device="cuda")
            x = s[new][b, :count].double()
            amax = x.abs().amax(-1)
            sc = torch.exp2(torch.floor(torch.log2(amax.clamp_min(2.0 ** -100) / E4M3_MAX)) - 1)
            sc = torch.where(E4M3_MAX * sc < amax, 2 * sc, sc)
            sc = torch.where(E4M3_MAX * sc < amax, 2 * sc, sc)
            sc = torch.where(amax > 0, sc, torch.ones_like(sc))
            page, row = s["table"][b].long()[at // R], at % R
            values[page, :, row] = _e4m3_nearest(x / sc[..., None])
            scale[page, :, row] = sc
        out[pool], out[scales] = values, scale
    return out


def _exact_rows(s, b, h, n):
    got = []
    for which, scale in (("K", "ks"), ("V", "vs")):
        x, sc = s[which], s.get(scale)
        if s["table"] is None:
            x, sc = x[b, h, :n], None if sc is None else sc[b, h, :n]
        else:
            pages = s["table"][b, : _ceil(n, x.shape[2])].long()
            x = x[:, h].view(torch.uint8)[pages].view(x.dtype).reshape(-1, D)[:n]
            sc = None if sc is None else sc[:, h][pages].reshape(-1)[:n]
        got.append(x.double() if sc is None else x.double() * sc.double()[:, None])
    return got


def _exact_decode(case, seed):
    s = prepare(case, seed)
    B, H, G = case["B"], case["H"], case["G"]
    out = torch.zeros((B, H * G, D), dtype=torch.float64, device="cuda")
    for b in range(B):
        n = int(s["lengths"][b])
        for h in range(H):
            if n == 0:
                continue
            K, V = _exact_rows(s, b, h, n)
            q = s["q"][b, h * G:(h + 1) * G].double()
            if case["op"] == "dense8":
                out[b, h * G:(h + 1) * G] = torch.softmax(q @ K.T / math.sqrt(D), -1) @ V
                continue
            w = D // 2
            lam = s["lam"].double()
            weight = math.exp(float(lam[0] @ lam[1])) - math.exp(float(lam[2] @ lam[3])) + s["lambda_init"]
            p = torch.softmax(q[:, :w] @ K[:, :w].T / math.sqrt(w), -1)
            p = p - weight * torch.softmax(q[:, w:] @ K[:, w:].T / math.sqrt(w), -1)
            o = p @ V
            o = o / torch.sqrt((o * o).mean(-1, keepdim=True) + s["eps"])
            out[b, h * G:(h + 1) * G] = o * s["gamma"].double() * (1 - s["lambda_init"])
    return out


def exact(case, seed):
    if case["op"] == "store":
        return _exact_store(case, seed)
    if case["op"] in ("dense8", "diff"):
        return _exact_decode(case, seed)
    return None  # page numbers and copied bits: whole numbers, equal or wrong
