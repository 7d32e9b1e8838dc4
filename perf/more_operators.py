"""Measured cases of what a sequence's tokens go through around the decode attention: rotary
positions, an int8 cache with a scale per block of tokens and head, the attention that reads it, and
cross attention.  Inputs, the plain form of each operator in elementary torch operations, and the
calls of this package (`own`).

  rope    queries and keys of new tokens turned by their positions, keys and values into the cache
  store   new keys and values rounded to int8 with a scale per block of tokens and head, into a
          cache's pages, and the same rows read back as every later attention sees them
  dense   full-scan decode attention over such a cache, one new token per sequence
  cross   attention of several query tokens, or of one, to keys and values of another length
"""
import math

import torch

own = False

D = 128          # row of a cache
I8_MAX = 127.0
LEAST = 2.0 ** -126  # the smallest scale of a block


# ------------------------------------------------------------------------------- the cases

def listed():
    return [
        # a decode step's new token of each sequence of a batch, all of the head turned: latency
        dict(name="rope-step", op="rope", B=8, H=8, G=4, T=1, n=4096, page=64, ragged=False, cache="bf16", block=64,
             rot=128, interleaved=False, scale="none"),
        # prompts of different lengths into an int8 cache, half of the head turned in pairs of neighbours
        dict(name="rope-prompt", op="rope", B=4, H=8, G=4, T=8191, n=4096, page=64, ragged=True, cache="i8", block=64,
             rot=64, interleaved=True, scale="linear"),
        # a chunk of a prompt that stands behind 1M tokens, in 16-row pages
        dict(name="rope-far", op="rope", B=1, H=8, G=5, T=4096, n=1048576, page=16, ragged=False, cache="bf16", block=16,
             rot=128, interleaved=False, scale="yarn"),
        # a decode step's new token of each sequence of a batch: latency
        dict(name="store-step", op="store", B=8, H=8, T=1, n=4096, page=64, ragged=False, block=64),
        # prompts of different lengths written into pages behind what is there
        dict(name="store-prompt", op="store", B=4, H=8, T=8191, n=4096, page=64, ragged=True, block=32),
        # a short chat in small pages: latency
        dict(name="dense-1000", op="dense", B=1, H=8, G=4, n=1000, page=16, ragged=False, block=16, out="f32"),
        # a batch of sequences between 16K and 64K with a KV head per query head
        dict(name="dense-varlen", op="dense", B=8, H=32, G=1, n=65536, page=64, ragged=True, block=64, out="bf16"),
        # one sequence of 1M tokens in a contiguous cache
        dict(name="dense-1m", op="dense", B=1, H=8, G=4, n=1048576, page=0, ragged=False, block=128, out="f32"),
        # one new token of each sequence to a short encoder's states: latency
        dict(name="cross-step", op="cross", B=8, H=8, G=4, T=1, n=1500, page=0, ragged=True),
        # prompts of a decoder to states of 1500 rows, a KV head per query head
        dict(name="cross-prompt", op="cross", B=8, H=16, G=1, T=500, n=1500, page=0, ragged=True),
        # a few query tokens of each sequence to 128K rows in pages
        dict(name="cross-few", op="cross", B=4, H=8, G=5, T=16, n=131072, page=64, ragged=False),
        # a long prompt to a long document
        dict(name="cross-long", op="cross", B=1, H=8, G=4, T=4096, n=32768, page=0, ragged=False),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["rope", "store", "dense", "cross"])
    page = rng.choice([16, 32, 64, 128])
    block = rng.choice([b for b in (16, 32, 64, 128) if b <= page])
    if op in ("rope", "store"):
        H, G = rng.choice([1, 2, 4, 8]), rng.choice([1, 2, 3, 4, 5, 8])
        B = _log(rng, 1, 32)
        T = _log(rng, 1, max(1, min(8191, 131072 // (B * H))))
        case = dict(op=op, B=B, H=H, T=T, n=_log(rng, 1, 4096), page=page, ragged=rng.random() < 0.5, block=block)
        if op == "rope":
            case |= dict(G=G, cache=rng.choice(["bf16", "i8"]), rot=rng.choice([16, 32, 48, 64, 80, 96, 128]),
                         interleaved=rng.random() < 0.5, scale=rng.choice(["none", "linear", "yarn"]))
        return case
    if op == "dense":
        H = rng.choice([1, 2, 4, 8, 32])
        G = rng.choice([1, 2, 3, 4, 5, 7, 8, 12, 16])
        B = _log(rng, 1, 16)
        n = _log(rng, 1, min(1 << 20, (1 << 22) // (B * H)))
        return dict(op=op, B=B, H=H, G=G, n=n, page=rng.choice([0, page]), ragged=rng.random() < 0.5, block=block,
                    out=rng.choice(["f32", "bf16"]))
    H, G = rng.choice([1, 2, 4, 8, 16]), rng.choice([1, 2, 3, 4, 5, 8])
    B = _log(rng, 1, 8)
    n = _log(rng, 1, min(131072, (1 << 22) // (B * H)))
    T = _log(rng, 1, max(1, min(4096, (1 << 31) // (B * H * G * n))))
    return dict(op=op, B=B, H=H, G=G, T=T, n=n, page=rng.choice([0, page]), ragged=rng.random() < 0.5)


# ------------------------------------------------------------------------------ the inputs

def _ceil(a, b):
    return -(-a // b)


def _lengths(case, gen, lo, hi, count):
    """int32 lengths on the device: hi each, or spread over [lo, hi] when the batch is ragged."""
    if not case["ragged"]:
        return torch.full((count,), hi, dtype=torch.int32, device="cuda")
    return torch.randint(lo, hi + 1, (count,), generator=gen, device="cuda", dtype=torch.int32)


def _keys(gen, slabs, H, rows):
    """bf16 [slabs, H, rows, D] keys around 64 centres of their head, as attention keys cluster."""
    centres = torch.randn((H, 64, D), generator=gen, device="cuda")
    z = torch.randint(0, 64, (slabs, H, rows), generator=gen, device="cuda")
    k = torch.randn((slabs, H, rows, D), generator=gen, device="cuda").mul_(0.5)
    k += centres[torch.arange(H, device="cuda")[None, :, None], z]
    return k.bfloat16(), centres


def _quantised(x, block):
    """(int8 codes, fp32 scale of each block of `block` rows) of rows [..., n, D]."""
    pad = -x.shape[-2] % block
    f = torch.nn.functional.pad(x.float(), (0, 0, 0, pad)).unflatten(-2, (-1, block))
    scale = (f.abs().amax((-1, -2)) / I8_MAX).clamp_min(LEAST)
    code = torch.round(f / scale[..., None, None]).clamp(-I8_MAX, I8_MAX).to(torch.int8)
    return code.flatten(-3, -2)[..., : x.shape[-2], :].contiguous(), scale


def _frequencies(case):
    """Radians per position of each pair of dimensions, and the factor of the turned part."""
    rot, base = case["rot"], 500000.0
    i = torch.arange(rot // 2, dtype=torch.float64, device="cuda")
    f = base ** (-2 * i / rot)
    if case["scale"] == "linear":
        return f / 4, 1.0
    if case["scale"] == "yarn":  # far turns interpolated, near ones kept, between 1 and 32 turns of 32K positions
        def dim(turns):
            return rot * math.log(32768 / (2 * math.pi * turns)) / (2 * math.log(base))
        lo, hi = max(math.floor(dim(32)), 0), min(math.ceil(dim(1)), rot - 1)
        keep = 1 - ((i - lo) / max(hi - lo, 0.001)).clamp(0, 1)
        return f / 32 * (1 - keep) + f * keep, 0.1 * math.log(32) + 1
    return f, 1.0


def _rows_new(gen, case, heads):
    x = torch.randn((case["B"], case["T"], heads, D), generator=gen, device="cuda")
    x *= torch.exp(0.3 * torch.randn((case["B"], case["T"], heads, 1), generator=gen, device="cuda"))
    return x.bfloat16()


def _prepare_store(case, gen):
    B, H, T, R, n = case["B"], case["H"], case["T"], case["page"], case["n"]
    pos = _lengths(case, gen, n // 2, n, B)
    count = _lengths(case, gen, T // 2, T, B)
    pps = _ceil(n + T, R)
    table = torch.randperm(B * pps, generator=gen, device="cuda").int().view(B, pps)
    G = case.get("G", 0)
    qkv = _rows_new(gen, case, (G + 2) * H)  # one fused projection's output
    s = dict(case=case, table=table, pos=pos, count=count, q=qkv[:, :, : G * H], k_new=qkv[:, :, G * H:(G + 1) * H],
             v_new=qkv[:, :, (G + 1) * H:])
    old = [torch.randn((B * pps, H, R, D), generator=gen, device="cuda", dtype=torch.bfloat16) for _ in range(2)]
    if case.get("cache", "i8") == "bf16":
        s["K"], s["V"] = old
    else:
        s["K"], s["ks"] = _quantised(old[0], case["block"])
        s["V"], s["vs"] = _quantised(old[1], case["block"])
    if case["op"] == "rope":
        s["freq"], s["factor"] = _frequencies(case)
    return s


def _tokens(s):
    """(b, t, position) of the new tokens."""
    T = s["k_new"].shape[1]
    b, t = torch.nonzero(torch.arange(T, device="cuda") < s["count"][:, None], as_tuple=True)
    return b, t, s["pos"].long()[b] + t


def _paged(gen, B, n, R):
    pps = _ceil(n, R)
    return torch.randperm(B * pps, generator=gen, device="cuda").int().view(B, pps)


def _prepare_attend(case, gen):
    B, H, G, n, R = case["B"], case["H"], case["G"], case["n"], case["page"]
    T = case.get("T", 1)
    table = _paged(gen, B, n, R) if R else None
    K, centres = _keys(gen, *((table.numel(), H, R) if R else (B, H, n)))
    V = torch.randn(K.shape, generator=gen, device="cuda").bfloat16()
    pick = torch.randint(0, 64, (B, T, H, G), generator=gen, device="cuda")
    q = 0.5 * centres[torch.arange(H, device="cuda")[None, None, :, None], pick]
    q = (q + 0.5 * torch.randn((B, T, H, G, D), generator=gen, device="cuda")).view(B, T, H * G, D).bfloat16()
    s = dict(case=case, lengths=_lengths(case, gen, max(1, n // 4), n, B), table=table, q=q, K=K, V=V)
    if case["op"] == "dense":
        s["q"] = q[:, 0].contiguous()
        s["K"], s["ks"] = _quantised(K, case["block"])
        s["V"], s["vs"] = _quantised(V, case["block"])
    return s


def prepare(case, seed):
    gen = torch.Generator(device="cuda").manual_seed(seed)
    make = dict(rope=_prepare_store, store=_prepare_store, dense=_prepare_attend, cross=_prepare_attend)
    return make[case["op"]](case, gen)


# -------------------------------------------------------------------------- the plain forms

def _turned(x, cos, sin, rot, interleaved):
    """fp32 rows x [..., heads, D] with their first `rot` dimensions turned; cos, sin [..., 1, rot / 2]."""
    if interleaved:
        a, b = x[..., 0:rot:2], x[..., 1:rot:2]
        y = torch.stack((a * cos - b * sin, b * cos + a * sin), -1).flatten(-2)
    else:
        a, b = x[..., : rot // 2], x[..., rot // 2: rot]
        y = torch.cat((a * cos - b * sin, b * cos + a * sin), -1)
    return torch.cat((y, x[..., rot:]), -1)


def _plain_block_store(s, which, scales, b, p, x):
    """Rows x [m, H, D] (fp32) to positions p of sequences b.  A block's scale only grows while rows are
    added behind those it holds, whose codes are then rounded anew."""
    pool, scale, block, table = s[which], s[scales], s["case"]["block"], s["table"].long()
    B, pps = table.shape
    H, R = pool.shape[1], pool.shape[2]
    per = R // block
    blk = p // block
    amax = torch.zeros((B * pps * per, H), device="cuda")
    amax.scatter_reduce_(0, (b * pps * per + blk)[:, None].expand(-1, H), x.abs().amax(-1), "amax")
    pages = scale[table].transpose(2, 3).reshape(B * pps * per, H)  # the scales in the order of the sequences' blocks
    start = s["pos"].long()
    first = torch.arange(B, device="cuda") * pps * per + (start // block).clamp_max(pps * per - 1)
    held = ((start % block) > 0) & (s["count"] > 0)  # the first block holds rows
    was = torch.zeros_like(pages)
    was[first] = torch.where(held[:, None], pages[first], 0.0)
    new = torch.maximum(torch.maximum(was, amax / I8_MAX), torch.full_like(was, LEAST))
    # rows that the first block holds
    at = (start // block * block)[:, None] + torch.arange(block, device="cuda")
    ob, ot = torch.nonzero(held[:, None] & (at < start[:, None]), as_tuple=True)
    op = at[ob, ot]
    ratio = was[first[ob]] / new[first[ob]]
    codes = pool[table[ob, op // R], :, op % R].float()
    pool[table[ob, op // R], :, op % R] = torch.round(codes * ratio[..., None]).to(torch.int8)
    # the new rows
    mine = new[b * pps * per + blk]
    code = torch.round(x * (1.0 / mine)[..., None]).clamp(-I8_MAX, I8_MAX).to(torch.int8)
    pool[table[b, p // R], :, p % R] = code
    scale[table[b, p // R], :, p % R // block] = mine


def _plain_load(s, which, scales, b, t, p):
    """bf16 [B, T, H, D] rows of the new tokens, zeros behind a sequence's last."""
    pool, table, block = s[which], s["table"].long(), s["case"]["block"]
    R = pool.shape[2]
    page = table[b, p // R]
    out = torch.zeros(s["k_new"].shape, device="cuda", dtype=torch.bfloat16)
    out[b, t] = (pool[page, :, p % R].float() * s[scales][page, :, p % R // block][..., None]).bfloat16()
    return out


def _plain_store(s):
    b, t, p = _tokens(s)
    _plain_block_store(s, "K", "ks", b, p, s["k_new"][b, t].float())
    _plain_block_store(s, "V", "vs", b, p, s["v_new"][b, t].float())
    return dict(k=_plain_load(s, "K", "ks", b, t, p), v=_plain_load(s, "V", "vs", b, t, p), ks=s["ks"], vs=s["vs"])


def _plain_rope(s):
    case = s["case"]
    b, t, p = _tokens(s)
    angle = p.double()[:, None] * s["freq"]  # (1M positions: 32 bits would leave a tenth of a radian)
    cos, sin = (f(angle).float()[:, None] * s["factor"] for f in (torch.cos, torch.sin))
    turn = (cos, sin, case["rot"], case["interleaved"])
    q = torch.zeros(s["q"].shape, device="cuda", dtype=torch.bfloat16)
    q[b, t] = _turned(s["q"][b, t].float(), *turn).bfloat16()
    k = _turned(s["k_new"][b, t].float(), *turn).bfloat16()  # the key that a cache of bf16 rows would hold
    if case["cache"] == "i8":
        _plain_block_store(s, "K", "ks", b, p, k.float())
        _plain_block_store(s, "V", "vs", b, p, s["v_new"][b, t].float())
        return dict(q=q, k=_plain_load(s, "K", "ks", b, t, p), v=_plain_load(s, "V", "vs", b, t, p))
    R = s["K"].shape[2]
    page = s["table"].long()[b, p // R]
    s["K"][page, :, p % R] = k
    s["V"][page, :, p % R] = s["v_new"][b, t]
    return dict(q=q, K=s["K"], V=s["V"])


def _plain_rows(s, which, scale):
    """fp32 [B, H, n, D] rows of the cache in order."""
    x, table = s[which], s["table"]
    if scale in s:
        x = x.float() * s[scale].repeat_interleave(s["case"]["block"], -1)[..., : x.shape[2], None]
    if table is not None:
        x = x[table.long()].transpose(1, 2).flatten(2, 3)  # [B, pages, H, R, D] -> [B, H, pages * R, D]
    return x.float()


def _plain_attention(q, K, V, lengths):
    """softmax(q K^T / sqrt D) V over each sequence's rows; zeros where there are none."""
    logit = torch.matmul(q, K.transpose(-1, -2)).mul_(1 / math.sqrt(D))
    seen = torch.arange(K.shape[2], device="cuda") < lengths.view(-1, 1, 1, 1)
    logit.masked_fill_(~seen, float("-inf"))
    w = logit.sub_(logit.amax(-1, keepdim=True)).exp_()
    w.masked_fill_(~seen, 0.0)
    total = w.sum(-1, keepdim=True)
    return torch.matmul(w, V) / torch.where(total > 0, total, 1.0)


def _out_type(case):
    return torch.float32 if case["out"] == "f32" else torch.bfloat16


def _plain_dense(s):
    B, H, G = (s["case"][k] for k in ("B", "H", "G"))
    K, V = _plain_rows(s, "K", "ks"), _plain_rows(s, "V", "vs")
    out = _plain_attention(s["q"].float().view(B, H, G, D), K, V, s["lengths"])
    return out.view(B, H * G, D).to(_out_type(s["case"]))


def _plain_cross(s):
    B, T, H, G = (s["case"][k] for k in ("B", "T", "H", "G"))
    K, V = _plain_rows(s, "K", "ks"), _plain_rows(s, "V", "vs")
    q = s["q"].float().view(B, T, H, G, D).permute(0, 2, 1, 3, 4).reshape(B, H, T * G, D)
    out = _plain_attention(q, K, V, s["lengths"])
    return out.view(B, H, T, G, D).permute(0, 2, 1, 3, 4).reshape(B, T, H * G, D).bfloat16()


# --------------------------------------------------------------------- this package's calls

def _own_cache(s):
    """The cache object that a program makes once, when it lays its cache out."""
    if "own_cache" not in s:
        import serving_mog_decode_gb300 as mog
        K, V, table = s["K"], s["V"], s["table"]
        if "ks" not in s:
            s["own_cache"] = (K, V) if table is None else (mog.PagedKV(K, V, table, K.shape[2]), None)
        elif table is None:
            s["own_cache"] = mog.KVI8(K, V, s["ks"], s["vs"], s["case"]["block"]), None
        else:
            s["own_cache"] = mog.PagedKVI8(K, V, s["ks"], s["vs"], table, K.shape[2], s["case"]["block"]), None
    return s["own_cache"]


def _own_load(s, K, V):
    """The new tokens' rows; what lies behind a sequence's last stays as the caller made it: zeros."""
    import serving_mog_decode_gb300 as mog
    k, v = torch.zeros((2,) + s["k_new"].shape, device="cuda", dtype=torch.bfloat16)
    return mog.kv_load(K, V, s["pos"], s["count"], k, v)


def _own_store(s):
    import serving_mog_decode_gb300 as mog
    K, V = _own_cache(s)
    mog.kv_store(K, V, s["pos"], s["count"], s["k_new"], s["v_new"])
    k, v = _own_load(s, K, V)
    return dict(k=k, v=v, ks=s["ks"], vs=s["vs"])


def _own_rope(s):
    import serving_mog_decode_gb300 as mog
    case = s["case"]
    if "turn" not in s:  # (a program keeps it for all its layers and steps)
        s["turn"] = mog.Rope(case["rot"], inv_freq=s["freq"], interleaved=case["interleaved"], factor=s["factor"])
    K, V = _own_cache(s)
    q = torch.zeros(s["q"].shape, device="cuda", dtype=torch.bfloat16)
    mog.rope_store(K, V, s["pos"], s["count"], s["q"], s["k_new"], s["v_new"], s["turn"], q_out=q)
    if case["cache"] == "i8":
        k, v = _own_load(s, K, V)
        return dict(q=q, k=k, v=v)
    return dict(q=q, K=s["K"], V=s["V"])


def _own_dense(s):
    import serving_mog_decode_gb300 as mog
    K, V = _own_cache(s)
    out = torch.empty(s["q"].shape, dtype=_out_type(s["case"]), device="cuda")
    return mog.dense_decode(K, V, s["lengths"], s["case"]["n"], s["q"], out=out)


def _own_cross(s):
    import serving_mog_decode_gb300 as mog
    K, V = _own_cache(s)
    return mog.cross_attend(K, V, s["lengths"], s["case"]["n"], s["q"])


def run(state):
    op = state["case"]["op"]
    if own:
        return dict(rope=_own_rope, store=_own_store, dense=_own_dense, cross=_own_cross)[op](state)
    return dict(rope=_plain_rope, store=_plain_store, dense=_plain_dense, cross=_plain_cross)[op](state)


# ------------------------------------------------------------------------ what a pass needs

def work(case):
    """Expected bytes and operations over the distribution of ragged lengths."""
    op, B, H = case["op"], case["B"], case["H"]
    if op in ("rope", "store"):
        tokens = B * (0.75 if case["ragged"] and case["T"] > 1 else 1) * case["T"]
        G = case.get("G", 0)
        i8 = case.get("cache", "i8") == "i8"
        kv = 2 * H * (2 * D + (D + 4 / case["block"] + 2 * D if i8 else 2 * D))  # read; the cache's row; read back
        ops = 3 * case.get("rot", 0) * (G + 1) * H + (2 * H * 4 * D if i8 else 0)
        return dict(bytes=tokens * (kv + G * H * 4 * D), flops=tokens * ops)
    G, T = case["G"], case.get("T", 1)
    rows = B * H * case["n"] * (0.625 if case["ragged"] else 1)
    if op == "dense":
        out = 4 if case["out"] == "f32" else 2
        return dict(bytes=2 * rows * (D + 4 / case["block"]) + B * H * G * D * (2 + out), flops=4 * rows * G * D)
    return dict(bytes=2 * rows * 2 * D + B * T * H * G * D * 4, flops=4 * rows * T * G * D)


# ------------------------------------------------ the definitions, in 64 bits, sequence by sequence

def _exact_blocks(new, old_scale, start, block):
    """Values that int8 blocks stand for, of rows new [m, H, D] (64 bits) from position `start` on,
    the block of which has the scales old_scale [H] if it holds rows; and the blocks' scales."""
    values, scales, m, at = [], [], new.shape[0], 0
    while at < m:
        room = block - (start + at) % block
        x = new[at:at + room]
        sc = (x.abs().amax((0, 2)) / I8_MAX).clamp_min(LEAST)
        if at == 0 and start % block:
            sc = torch.maximum(sc, old_scale)
        code = torch.round(x / sc[:, None]).clamp(-I8_MAX, I8_MAX)
        values.append(code * sc[:, None])
        scales.append(sc)
        at += room
    return torch.cat(values) if values else new, scales


def _exact_store(case, seed):
    s = prepare(case, seed)
    R, block, shape = case["page"], case["block"], s["k_new"].shape
    out = {}
    if case["op"] == "rope":
        out["q"] = torch.zeros(s["q"].shape, dtype=torch.float64, device="cuda")
    i8 = "ks" in s
    for pool, scales, new, name in (("K", "ks", "k_new", "k"), ("V", "vs", "v_new", "v")):
        read = torch.zeros(shape, dtype=torch.float64, device="cuda")
        held = s[scales].double() if i8 else s[pool].double()
        for b in range(case["B"]):
            count, start = int(s["count"][b]), int(s["pos"][b])
            x = s[new][b, :count].double()
            at = torch.arange(start, start + count, device="cuda")
            page = s["table"][b].long()[at // R]
            if case["op"] == "rope":
                z = torch.polar(torch.full((), s["factor"], dtype=torch.float64, device="cuda"),
                                at.double()[:, None] * s["freq"])
                if name == "k":
                    out["q"][b, :count] = _exact_turn(s["q"][b, :count].double(), z, case)
                    x = _exact_turn(x, z, case).bfloat16().double()
            if not i8:
                held[page, :, at % R] = x
                continue
            first = s["table"][b, min(start // R, s["table"].shape[1] - 1)].long()
            read[b, :count], sc = _exact_blocks(x, held[first, :, start % R // block], start, block)
            for i, one in enumerate(sc):
                p = start // block + i
                held[s["table"][b, p * block // R].long(), :, p * block % R // block] = one
        if not i8:
            out[pool] = held
            continue
        out[name] = read
        if case["op"] == "store":
            out[scales] = held
    return out


def _exact_turn(x, z, case):
    """Rows x [m, heads, D] in 64 bits, their pairs turned by the complex numbers z [m, rot / 2]."""
    rot, out = case["rot"], x.clone()
    part = x[..., :rot]
    pair = part.unflatten(-1, (-1, 2)) if case["interleaved"] else part.unflatten(-1, (2, -1)).transpose(-1, -2)
    turned = torch.view_as_real(torch.view_as_complex(pair.contiguous()) * z[:, None])
    out[..., :rot] = (turned if case["interleaved"] else turned.transpose(-1, -2)).flatten(-2)
    return out


def _exact_rows(s, b, h, n):
    got = []
    for which, scale in (("K", "ks"), ("V", "vs")):
        x, sc = s[which], s.get(scale)
        if s["table"] is None:
            x, sc = x[b, h, :n], None if sc is None else sc[b, h]
        else:
            pages = s["table"][b, : _ceil(n, x.shape[2])].long()
            x, sc = x[:, h][pages].reshape(-1, D)[:n], None if sc is None else sc[:, h][pages].reshape(-1)
        x = x.double()
        got.append(x if sc is None else x * sc.double()[torch.arange(n, device="cuda") // s["case"]["block"]][:, None])
    return got


def _exact_attend(case, seed):
    s = prepare(case, seed)
    B, H, G, T = case["B"], case["H"], case["G"], case.get("T", 1)
    if case["n"] * B * H * G * T > 1 << 33:
        return None
    q = s["q"].view(B, T, H, G, D)
    out = torch.zeros(q.shape, dtype=torch.float64, device="cuda")
    for b in range(B):
        n = int(s["lengths"][b])
        for h in range(H):
            K, V = _exact_rows(s, b, h, n)
            logits = q[b, :, h].reshape(-1, D).double() @ K.T / math.sqrt(D)
            out[b, :, h] = (torch.softmax(logits, -1) @ V).view(T, G, D)
    return out.view(s["q"].shape)


def exact(case, seed):
    return _exact_store(case, seed) if case["op"] in ("rope", "store") else _exact_attend(case, seed)
