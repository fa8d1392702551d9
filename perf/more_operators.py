"""Cases and reference forms of rotary positions, scored attention, eviction and adapters.

Five kinds of work, each in a plain form (elementary torch operations in 32
bits, angles in 64, rounded once at the end) and, with ``own`` true, as the
calls that a user makes of the package:

  rotate  rotary positions on the heads of many tokens
  append  the same on a decode step's queries and keys, keys and values going to
          a paged cache
  score   tree attention over a paged cache that also adds up, for each cached
          key, the attention weight that it has received
  evict   each kv head keeps the keys with the largest weights so far, beside
          the first and the last ones, in their order, on other pages
  lora    y = W x + s B (A x): 4-bit rows that all tokens share, and each
          token's own low-rank adapter

The 4-bit rows are the package's format: kp/2 bytes of codes (kp = k rounded up
to a multiple of 128), then fp16 group scales, zero padded.  Weight i is
(code - 8) * scale[i // group]; in each block of 128 weights (16 words of 32
bits) word 4t+j holds weights 32j+8t .. 32j+8t+7, and weight 2p+h of a word is
the nibble at bit 16h+4p.  Weights past k have code 8.
"""
import math

import torch

own = False


# ------------------------------------------------------------------ cases --
def listed():
    return [
        # queries and keys of one decoded token of the 70B shape: latency
        dict(name="rotate one token", kind="rotate", T=1, heads=72, D=128, rot=128, layout="half", scaling="none",
             dtype="f16", far=40000, spare=8),
        # a whole prompt of the 70B shape under a context extended 8 times, slices of the joint projection
        dict(name="rotate prompt 8192", kind="rotate", T=8192, heads=72, D=128, rot=128, layout="half", scaling="yarn",
             dtype="f16", far=32000, spare=8),
        # an fp32 layer that turns a part of odd width of its heads, neighbours paired, positions past a million
        dict(name="rotate part f32 pairs", kind="rotate", T=1111, heads=36, D=80, rot=36, layout="pairs",
             scaling="linear", dtype="f32", far=1500000, spare=0),
        # a decode step of 32 requests of the 70B shape
        dict(name="append r32", kind="append", R=32, T=32, L=4096, hkv=8, grp=8, D=128, rot=128, layout="half",
             scaling="none", page=16, far=4096),
        # eight drafted tokens of a 64-wide, 128-headed model, a quarter of the head turned
        dict(name="append tree part", kind="append", R=3, T=24, L=700, hkv=8, grp=16, D=64, rot=16, layout="pairs",
             scaling="ntk", page=20, far=9000),
        # one new token after a short prompt, heads of their own
        dict(name="score short b1", kind="score", R=1, T=1, L=333, hkv=32, grp=1, D=128, page=16, ragged=False),
        # eight conversations of a batch, one token each
        dict(name="score ragged r8", kind="score", R=8, T=8, L=16001, hkv=8, grp=8, D=128, page=64, ragged=True),
        # sixteen drafted tokens of one long conversation
        dict(name="score long t16", kind="score", R=1, T=16, L=65500, hkv=8, grp=8, D=128, page=64, ragged=False),
        # a conversation of heads of their own brought back to a quarter
        dict(name="evict 4000 to 1000", kind="evict", R=1, L=4000, keep=1000, first=4, recent=256, hkv=32, D=128, page=16,
             ragged=False),
        # long conversations of different lengths, one of them still short, brought to 16384 keys
        dict(name="evict ragged r4", kind="evict", R=4, L=65500, keep=16384, first=4, recent=4096, hkv=8, D=128, page=64,
             ragged=True),
        # one token through a square projection with an adapter: latency
        dict(name="lora 7B square b1", kind="lora", m=4096, k=4096, B=1, group=128, rank=16, adapters=8, dtype="f16"),
        # 32 requests, most with an adapter of their own, through the widest projection of the 70B shape
        dict(name="lora 70B up b32", kind="lora", m=28672, k=8192, B=32, group=128, rank=64, adapters=24, dtype="f16"),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    kind = rng.choice(["rotate", "rotate", "append", "score", "score", "evict", "evict", "lora", "lora"])
    D = rng.choice([64, 80, 128])
    layout, scaling = rng.choice(["half", "pairs"]), rng.choice(["none", "linear", "ntk", "yarn"])
    rot = rng.choice([D, D, D // 2, 2 * rng.randint(1, D // 2)])
    if kind == "rotate":
        heads = rng.choice([1, 9, 36, 64, 72, rng.randint(2, 130)])
        T = min(_log(rng, 1, 20000), 8192 * 72 * 128 // (heads * D))
        return dict(kind=kind, T=T, heads=heads, D=D, rot=rot, layout=layout, scaling=scaling,
                    dtype=rng.choice(["f16", "f16", "f32"]) if T * heads * D <= 4096 * 72 * 128 else "f16",
                    far=_log(rng, 100, 2000000), spare=rng.choice([0, 0, 8]))
    hkv = rng.choice([1, 2, 8, 32])
    page = rng.choice([16, 20, 64, 256])
    if kind == "evict":
        R = rng.choice([1, 1, 2, 5, 16])
        L = _log(rng, 2, 200000 // (R * max(1, hkv // 8)))
        keep = max(1, int(L * rng.uniform(0.05, 0.9)))
        first = min(keep, rng.choice([0, 0, 4]))
        return dict(kind=kind, R=R, L=L, keep=keep, first=first, recent=int((keep - first) * rng.choice([0, 0.1, 0.5])),
                    hkv=hkv, D=D, page=page, ragged=rng.random() < 0.5)
    if kind == "lora":
        k = 8 * _log(rng, 16, 1536)
        m = max(1, min(_log(rng, 64, 28672), 28672 * 8192 // k))
        return dict(kind=kind, m=m, k=k, B=rng.choice([1, 1, 2, rng.randint(3, 8), rng.randint(9, 32)]),
                    group=rng.choice([32, 64, 128]), rank=rng.choice([8, 16, 16, 24, 32, 64]), adapters=rng.randint(1, 24),
                    dtype=rng.choice(["f16", "f16", "f32"]))
    grp = rng.choice([1, 1, 4, 7, 8, 16]) if hkv < 32 else 1
    R = rng.choice([1, 1, 2, 5, 16, 32])
    T = rng.randint(R, 32) if kind == "append" or rng.random() < 0.5 else R
    L = _log(rng, 1, 60000 // (R * max(1, hkv // 8)) + 2)
    if kind == "append":
        return dict(kind=kind, R=R, T=T, L=L, hkv=hkv, grp=grp, D=D, rot=rot, layout=layout, scaling=scaling, page=page,
                    far=_log(rng, 100, 2000000))
    return dict(kind=kind, R=R, T=T, L=L, hkv=hkv, grp=grp, D=D, page=page, ragged=rng.random() < 0.5)


def _size(case):
    return 2 if case["dtype"] == "f16" else 4


def work(case):
    kind = case["kind"]
    if kind == "rotate":
        n = case["T"] * case["heads"]
        return {"bytes": 2 * n * case["D"] * _size(case), "flops": 3 * n * case["rot"]}
    if kind == "append":
        n = case["T"] * case["hkv"] * (case["grp"] + 1)
        return {"bytes": 4 * case["D"] * (n + case["T"] * case["hkv"]), "flops": 3 * n * case["rot"]}
    if kind == "lora":
        m, k, B, r = case["m"], case["k"], case["B"], case["rank"]
        used = len(set(_adapters(case)) - {-1})
        each = sum(a >= 0 for a in _adapters(case))
        return {"bytes": m * k * (0.5 + 2.0 / case["group"]) + used * (m + k) * r * _size(case) + B * (k * _size(case) + 4 * m),
                "flops": 2 * m * k * B + 2 * (m + k) * r * each}
    lens, begin = _requests(case)
    hkv, D = case["hkv"], case["D"]
    if kind == "evict":
        kept = sum(min(n, case["keep"]) for n in lens)
        return {"bytes": hkv * (4 * sum(lens) + kept * (8 * D + 12)), "flops": 0}
    T, grp = case["T"], case["grp"]
    seen = sum(lens[r] + begin[r + 1] - begin[r] for r in range(case["R"]))
    pairs = sum((begin[r + 1] - begin[r]) * (lens[r] + begin[r + 1] - begin[r]) for r in range(case["R"]))
    return {"bytes": hkv * seen * (4 * D + 8) + 4 * D * hkv * grp * T, "flops": (4 * D + 4) * hkv * grp * pairs}


# ----------------------------------------------------------------- inputs --
def _requests(case):
    """Cached lengths and token ranges of the requests: fixed by the case."""
    R, L = case["R"], case["L"]
    if case.get("ragged"):
        lens = [max(0, L * (r * 7 % R + 1) // R - 1 - r) for r in range(R)]
        if R > 2:
            lens[2] = min(lens[2], 3)                                      # a request that has only just begun
    else:
        lens = [max(0, L - r) for r in range(R)]
    T = case.get("T", 0)
    return lens, [T * r // R for r in range(R + 1)]


def _adapters(case):
    """Which adapter each token uses: some share one, some have none; fixed by the case."""
    if case["B"] == 1:
        return [case["adapters"] - 1]
    return [-1 if b % 11 == 5 else b * 5 % case["adapters"] for b in range(case["B"])]


_BASE, _FACTOR, _ORIGINAL = 10000.0, 8.0, 4096


def _frequencies(case):
    """Radians per position of each pair, in 64 bits, and what cos and sin are multiplied by."""
    rot = case["rot"]
    i = torch.arange(rot // 2, dtype=torch.float64)
    if case["scaling"] == "ntk":                                           # the base grows so that the slowest pair turns
        base = _BASE * _FACTOR ** (rot / (rot - 2)) if rot > 2 else _BASE  # as slowly as if positions were divided
        return base ** (-2 * i / rot), 1.0
    f = _BASE ** (-2 * i / rot)
    if case["scaling"] == "linear":
        return f / _FACTOR, 1.0
    if case["scaling"] == "yarn":
        # pairs that turn more than 32 times in the original context stay, those that turn less than once are divided
        at = [rot * math.log(_ORIGINAL / (2 * math.pi * n)) / (2 * math.log(_BASE)) for n in (32.0, 1.0)]
        low, high = max(math.floor(at[0]), 0), min(math.ceil(at[1]), rot - 1)
        ramp = ((i - low) / max(high - low, 0.001)).clamp(0, 1)
        return f * (1 - ramp) + f / _FACTOR * ramp, 0.1 * math.log(_FACTOR) + 1.0
    return f, 1.0


def _rotary(s, case):
    f, s["mul"] = _frequencies(case)
    s["freq"] = f.cuda()
    if own:
        import activation_sparse_ffn_predict_b200 as A
        s["A"] = A
        s["rot"] = A.Rotary(case["D"], case["rot"], base=_BASE, layout=case["layout"], scaling=case["scaling"],
                            factor=_FACTOR, original=_ORIGINAL)


def _pad(k):
    return -(-k // 128) * 128


def _row_bytes(k, group):
    scales = -(-_pad(k) // 512) * (512 // group) * 2
    return _pad(k) // 2 + -(-scales // 16) * 16


def _pack(w, group):
    """fp32 rows [m, k] as 4-bit rows [m, row_bytes] (uint8)."""
    m, k = w.shape
    kp = _pad(k)
    w = torch.nn.functional.pad(w, (0, kp - k)).view(m, kp // group, group)
    s = (w.abs().amax(-1) / torch.full((), 7.0, device=w.device)).half()
    sf = s.float().unsqueeze(-1)
    c = torch.where(sf > 0, torch.round(w / sf), torch.zeros_like(w)).clamp_(-8, 7).to(torch.int32).add_(8)
    c = c.view(m, kp // 128, 4, 4, 4, 2)                                   # block, j, t, p, h
    at = torch.tensor([[0, 16], [4, 20], [8, 24], [12, 28]], device=w.device, dtype=torch.int32)
    words = (c << at).sum((-1, -2), dtype=torch.int32)                     # nibbles do not overlap: a sum is an or
    out = torch.zeros(m, _row_bytes(k, group), dtype=torch.uint8, device=w.device)
    out[:, :kp // 2] = words.transpose(-1, -2).contiguous().view(torch.uint8).view(m, kp // 2)
    out[:, kp // 2:kp // 2 + 2 * (kp // group)] = s.contiguous().view(torch.uint8).view(m, -1)
    return out


def _packed_normal(m, k, std, group, gen):
    """Normal weights, packed a few thousand rows at a time."""
    step = max(1, (1 << 26) // k)
    return torch.cat([_pack(torch.randn(min(step, m - i), k, generator=gen, device="cuda") * std, group)
                      for i in range(0, m, step)])


def prepare(case, seed):
    gen = torch.Generator(device="cuda").manual_seed(seed)

    def normal(*shape):
        return torch.randn(*shape, generator=gen, device="cuda")

    def tables(need, spare, order=None):
        """Shuffled pages for requests of `need` pages each, and how many pages there are."""
        if order is None:
            order = torch.rand(sum(need) + spare, generator=gen, device="cuda").argsort().to(torch.int32)
        table = torch.zeros(len(need), max(need), dtype=torch.int32, device="cuda")
        at = 0
        for r, n in enumerate(need):
            table[r, :n] = order[at:at + n]
            at += n
        return table, order[at:]

    def ints(v):
        return torch.tensor(v, dtype=torch.int32, device="cuda")

    kind = case["kind"]
    s = dict(case=case, kind=kind)
    if kind == "rotate":
        dt = torch.float16 if case["dtype"] == "f16" else torch.float32
        T, heads, D = case["T"], case["heads"], case["D"]
        s["joint"] = normal(T, heads + case["spare"], D).to(dt)            # the joint projection's output
        s["x"] = s["joint"][:, :heads]
        s["y"] = torch.empty(T, heads, D, dtype=dt, device="cuda")
        s["pos"] = (torch.rand((), generator=gen, device="cuda") * case["far"]).int() + torch.arange(
            T, dtype=torch.int32, device="cuda")
        _rotary(s, case)
        return s
    if kind == "lora":
        dt = torch.float16 if case["dtype"] == "f16" else torch.float32
        m, k, B, r, n = (case[i] for i in ("m", "k", "B", "rank", "adapters"))
        s["data"] = _packed_normal(m, k, 1 / math.sqrt(k), case["group"], gen)
        s["x"] = normal(B, k).to(dt)
        s["down"] = (normal(n, r, k) / math.sqrt(k)).to(dt)
        s["up"] = (normal(n, m, r) / math.sqrt(r)).to(dt)
        s["scale"] = torch.rand(n, generator=gen, device="cuda") + 0.5
        s["which"] = ints(_adapters(case))
        s["y"] = torch.empty(B, m, device="cuda")
        if own:
            import activation_sparse_ffn_predict_b200 as A
            s["A"], s["mat"] = A, A.W4Matrix(s["data"], k, case["group"])
            s["lora"] = A.LoraSet(s["down"], s["up"], s["scale"])
            s["ws"] = A.Workspace.for_w4(s["mat"], B, lora=s["lora"])
        return s
    R, hkv, D, page = (case[i] for i in ("R", "hkv", "D", "page"))
    lens, begin = _requests(case)
    s["lens"], s["begin"] = ints(lens), ints(begin)
    s["longest"] = max(lens)
    if kind == "evict":
        keep = case["keep"]
        need = [-(-max(1, n) // page) for n in lens]
        fresh = [-(-max(1, min(n, keep)) // page) for n in lens]
        s["table"], rest = tables(need, sum(fresh) + 2)
        s["table_out"], _ = tables(fresh, 0, rest)
        pages, S = sum(need) + sum(fresh) + 2, max(1, s["longest"])
        s["k"], s["v"] = (normal(pages, page, hkv, D).half() for _ in range(2))
        # weights with a long tail; some keys were never looked at
        s["scores"] = torch.exp(2 * normal(R, hkv, S)) * (torch.rand(R, hkv, S, generator=gen, device="cuda") > 0.05)
        s["scores_out"] = torch.zeros(R, hkv, keep, device="cuda")
        s["kept"] = torch.zeros(R, hkv, keep, dtype=torch.int32, device="cuda")
        s["lens_out"] = torch.zeros(R, dtype=torch.int32, device="cuda")
        if own:
            import activation_sparse_ffn_predict_b200 as A
            s["A"], s["cache"] = A, A.KVCache(s["k"], s["v"])
            s["ws"] = A.Workspace.for_eviction(s["cache"])
        return s
    T, grp = case["T"], case["grp"]
    counts = [begin[r + 1] - begin[r] for r in range(R)]
    need = [-(-(lens[r] + counts[r]) // page) for r in range(R)]
    s["table"], _ = tables(need, 3)
    pages = sum(need) + 3
    s["k"], s["v"] = (normal(pages, page, hkv, D).half() for _ in range(2))
    if kind == "append":
        _rotary(s, case)
        s["qkv"] = normal(T, hkv * (grp + 2), D).half()                    # the joint projection's output
        s["q"], s["k_new"], s["v_new"] = s["qkv"].split([hkv * grp, hkv, hkv], 1)
        s["q_out"] = torch.empty(T, hkv * grp, D, dtype=torch.float16, device="cuda")
        s["pos"] = (torch.rand(T, generator=gen, device="cuda") * case["far"]).int()
        if own:
            A = s["A"]
            s["cache"] = A.KVCache(s["k"], s["v"])
            s["ws"] = A.Workspace.for_attention(s["cache"], hkv * grp, R, T)
        return s
    anc = []
    pick = torch.rand(T, generator=gen, device="cuda").tolist()
    for r in range(R):
        for i in range(counts[r]):
            t = begin[r] + i
            parent = int(pick[t] * (i + 1)) - 1                            # -1: the tree's root follows the prefix
            anc.append((1 << t) | (anc[begin[r] + parent] if parent >= 0 else 0))
    s["anc"] = ints([a - (1 << 32) if a >> 31 else a for a in anc])
    s["q"] = (normal(T, hkv * grp, D) * 1.5).half()
    s["o"] = torch.empty_like(s["q"])
    s["most"], s["tmax"] = max(lens[r] + counts[r] for r in range(R)), max(counts)
    # what a few earlier steps have left, on average
    s["scores"] = torch.rand(R, hkv, max(need) * page, generator=gen, device="cuda") * (8 * grp * s["tmax"] / s["most"])
    if own:
        import activation_sparse_ffn_predict_b200 as A
        s["A"], s["cache"] = A, A.KVCache(s["k"], s["v"])
        s["ws"] = A.Workspace.for_attention(s["cache"], hkv * grp, R, T, scored_pages=s["table"].shape[1])
    return s


# ------------------------------------------------------------ plain forms --
def _turn(x, pos, s):
    """x [T, heads, D] in fp32, turned."""
    c = s["case"]
    rot, half = c["rot"], c["rot"] // 2
    a = pos.double()[:, None] * s["freq"]
    cos, sin = ((g(a) * s["mul"]).float()[:, None] for g in (torch.cos, torch.sin))
    if c["layout"] == "half":
        u, w = x[..., :half], x[..., half:rot]
        return torch.cat([u * cos - w * sin, w * cos + u * sin, x[..., rot:]], -1)
    u, w = x[..., 0:rot:2], x[..., 1:rot:2]
    return torch.cat([torch.stack([u * cos - w * sin, w * cos + u * sin], -1).flatten(-2), x[..., rot:]], -1)


def _slots(s):
    """Page and slot of the call's tokens, and their requests."""
    T, page = s["case"]["T"], s["case"]["page"]
    tok = torch.arange(T, device="cuda")
    lens, begin = s["lens"].long(), s["begin"].long()
    req = (tok[:, None] >= begin[None, 1:]).sum(1)
    where = lens[req] + tok - begin[req]
    return s["table"][req, where // page].long(), where % page, req, tok - begin[req]


def _plain_append(s):
    pg, sl, _, _ = _slots(s)
    s["k"][pg, sl] = _turn(s["k_new"].float(), s["pos"], s).half()
    s["v"][pg, sl] = s["v_new"]
    s["q_out"][:] = _turn(s["q"].float(), s["pos"], s).half()
    return {"q": s["q_out"], "k": s["k"], "v": s["v"]}


def _plain_score(s):
    c = s["case"]
    hkv, grp, D, page, T, R = c["hkv"], c["grp"], c["D"], c["page"], c["T"], c["R"]
    lens, begin = s["lens"].long(), s["begin"].long()
    p = torch.arange(s["most"], device="cuda")
    j = p[None] - lens[:, None]                                            # [R, P] place among the drafted tokens
    own_t = (begin[1:] - begin[:-1])[:, None]
    drafted = (j >= 0) & (j < own_t)
    bit = torch.where(drafted, begin[:-1, None] + j, torch.zeros_like(j))
    i = torch.arange(s["tmax"], device="cuda")
    real = i[None] < own_t                                                 # [R, t]
    rows = torch.where(real, begin[:-1, None] + i[None], torch.zeros_like(i[None]))
    sees = (j < 0)[:, None] | (drafted[:, None] & (((s["anc"].long()[rows][:, :, None] >> bit[:, None]) & 1) > 0))
    sees = sees & real[:, :, None]
    page_of = s["table"].long()[:, p // page]
    k = s["k"][page_of, p % page].float().permute(0, 2, 3, 1)              # [R, hkv, D, P]
    v = s["v"][page_of, p % page].float().permute(0, 2, 1, 3)              # [R, hkv, P, D]
    q = s["q"].float().view(T, hkv, grp, D)[rows].permute(0, 2, 1, 3, 4).reshape(R, hkv, -1, D)
    z = ((q @ k) * (1 / math.sqrt(D))).view(R, hkv, -1, grp, s["most"]).masked_fill_(~sees[:, None, :, None], -math.inf)
    top = z.amax(-1, keepdim=True)
    e = torch.exp(z.sub_(torch.where(torch.isinf(top), torch.zeros_like(top), top)))
    total = e.sum(-1, keepdim=True)
    e = torch.where(total > 0, e / total, torch.zeros_like(e))
    o = (e.view(R, hkv, -1, s["most"]) @ v).view(R, hkv, -1, grp, D)
    _, _, req, place = _slots(s)
    s["o"][:] = o.permute(0, 2, 1, 3, 4)[req, place].reshape(T, hkv * grp, D).half()
    w, old = e.sum((2, 3)), s["scores"][:, :, :s["most"]]                  # [R, hkv, P]
    s["scores"][:, :, :s["most"]] = torch.where((j < 0)[:, None], old + w, torch.where(drafted[:, None], w, old))
    return {"o": s["o"], "scores": s["scores"]}


def _plain_evict(s):
    c = s["case"]
    keep, first, recent, page = c["keep"], c["first"], c["recent"], c["page"]
    n = s["lens"].long()[:, None, None]
    p = torch.arange(s["scores"].shape[2], device="cuda")
    held = (p < first) | (p >= n - recent)
    rank = torch.where(held, torch.full_like(s["scores"], math.inf), s["scores"])
    rank = torch.where(p < n, rank, torch.full_like(rank, -math.inf))
    best = torch.sort(rank, dim=-1, descending=True, stable=True).indices[..., :keep]
    m = min(keep, best.shape[-1])
    new = torch.minimum(s["lens"], torch.full_like(s["lens"], keep))
    j = torch.arange(m, device="cuda")
    there = j < new[:, None, None]                                         # [R, 1, m]
    best = torch.sort(torch.where(there, best, torch.full_like(best, p.numel())), -1).values
    old = torch.where(there, best, torch.zeros_like(best))
    s["kept"][..., :m] = torch.where(there, best.int(), s["kept"][..., :m])
    s["scores_out"][..., :m] = torch.where(there, s["scores"].gather(-1, old), s["scores_out"][..., :m])
    r, h, i = there.expand_as(best).nonzero(as_tuple=True)
    src, dst = best[r, h, i], i
    to, at = s["table_out"][r, dst // page].long(), s["table"][r, src // page].long()
    s["k"][to, dst % page, h] = s["k"][at, src % page, h]
    s["v"][to, dst % page, h] = s["v"][at, src % page, h]
    s["lens_out"][:] = new
    return {n: s[n] for n in ("k", "v", "kept", "scores_out", "lens_out")}


def _unpack(data, k, group):
    """fp32 rows [..., k] of 4-bit rows [..., row_bytes]."""
    kp = _pad(k)
    lead = data.shape[:-1]
    words = data[..., :kp // 2].contiguous().view(torch.int32).view(*lead, kp // 128, 4, 4).transpose(-1, -2).contiguous()
    at = torch.tensor([0, 16, 4, 20, 8, 24, 12, 28], device=data.device, dtype=torch.int32)
    c = ((words.unsqueeze(-1) >> at) & 15).sub_(8).float().view(*lead, kp // group, group)
    s = data[..., kp // 2:kp // 2 + 2 * (kp // group)].contiguous().view(torch.float16).float()
    return (c * s.unsqueeze(-1)).view(*lead, kp)[..., :k]


def _plain_lora(s):
    c = s["case"]
    x, a = s["x"].float(), s["which"].long()
    at = a.clamp(min=0)
    y = x @ _unpack(s["data"], c["k"], c["group"]).t()
    h = (s["down"][at].float() @ x[:, :, None])                            # [B, r, 1]
    d = (s["up"][at].float() @ h)[:, :, 0] * s["scale"][at][:, None]
    return y + torch.where(a[:, None] >= 0, d, torch.zeros_like(d))


def run(s):
    kind = s["kind"]
    if own:
        A = s["A"]
        if kind == "rotate":
            A.asf_rotary_apply(s["rot"], s["x"], s["pos"], s["y"])
            return s["y"]
        if kind == "append":
            A.asf_rotary_append(s["rot"], s["cache"], s["table"], s["lens"], s["begin"], s["pos"], s["q"], s["q_out"],
                                s["k_new"], s["v_new"], s["ws"])
            return {"q": s["q_out"], "k": s["k"], "v": s["v"]}
        if kind == "score":
            A.asf_tree_attention_scored(s["cache"], s["table"], s["lens"], s["begin"], s["q"], s["anc"], s["o"],
                                        s["scores"], s["ws"])
            return {"o": s["o"], "scores": s["scores"]}
        if kind == "evict":
            c = s["case"]
            A.asf_kv_evict(s["cache"], s["table"], s["lens"], s["scores"], c["keep"], s["table_out"], s["lens_out"],
                           s["scores_out"], s["kept"], s["ws"], first=c["first"], recent=c["recent"])
            return {n: s[n] for n in ("k", "v", "kept", "scores_out", "lens_out")}
        A.asf_w4_matmul_lora(s["mat"], s["lora"], s["which"], s["x"], s["y"], s["ws"])
        return s["y"]
    if kind == "rotate":
        s["y"][:] = _turn(s["x"].float(), s["pos"], s).to(s["y"].dtype)
        return s["y"]
    return {"append": _plain_append, "score": _plain_score, "evict": _plain_evict, "lora": _plain_lora}[kind](s)


# ------------------------------------------------------- 64-bit definition --
def _turned64(x, pos, case):
    """From the definition: pair j of a token at p, as a complex number, times mul e^(i p f_j)."""
    y, x, rot = x.double().clone(), x.double(), case["rot"]
    f, mul = _frequencies(case)
    j = torch.arange(rot // 2, device="cuda")
    a, b = (j, j + rot // 2) if case["layout"] == "half" else (2 * j, 2 * j + 1)
    angle = pos.double()[:, None] * f.cuda()
    z = torch.complex(x[..., a], x[..., b]) * torch.polar(torch.full_like(angle, mul), angle)[:, None]
    y[..., a], y[..., b] = z.real, z.imag
    return y


def _rows64(data, k, group):
    """float64 rows of 4-bit rows [m, row_bytes], weight by weight from the layout's description."""
    i = torch.arange(k, device=data.device)
    inside = i % 128
    j, t, e = inside // 32, inside % 32 // 8, inside % 8
    bit = 16 * (e % 2) + 4 * (e // 2)
    byte = (i // 128) * 64 + (4 * t + j) * 4 + bit // 8
    code = (data[:, byte].to(torch.int64) >> (bit % 8)) & 15
    first = _pad(k) // 2
    pair = data[:, first + 2 * (i // group)].to(torch.int64) + 256 * data[:, first + 2 * (i // group) + 1].to(torch.int64)
    expo, frac = (pair >> 10) & 31, pair & 1023                            # binary16, finite and not negative here
    scale = torch.where(expo > 0, torch.ldexp(1.0 + frac.double() / 1024, expo - 15), torch.ldexp(frac.double(), expo - 24))
    return (code - 8).double() * scale


def exact(case, seed):
    s = prepare(case, seed)
    kind = case["kind"]
    if kind == "rotate":
        return _turned64(s["x"], s["pos"], case)
    if kind == "lora":
        step = max(1, (1 << 25) // case["k"])
        x = s["x"].double()
        y = torch.cat([x @ _rows64(s["data"][a:a + step], case["k"], case["group"]).t() for a in range(0, case["m"], step)], 1)
        for b, a in enumerate(s["which"].tolist()):
            if a >= 0:
                y[b] += s["scale"][a].double() * (s["up"][a].double() @ (s["down"][a].double() @ x[b]))
        return y
    lens, begin = _requests(case)
    hkv, D, page = case["hkv"], case["D"], case["page"]
    if kind == "append":
        k, v = s["k"].double(), s["v"].double()
        turned = _turned64(s["k_new"], s["pos"], case)
        for r in range(case["R"]):
            for i, t in enumerate(range(begin[r], begin[r + 1])):
                a, b = divmod(lens[r] + i, page)
                k[s["table"][r, a], b], v[s["table"][r, a], b] = turned[t], s["v_new"][t].double()
        return {"q": _turned64(s["q"], s["pos"], case), "k": k, "v": v}
    if kind == "evict":
        first, recent, keep = case["first"], case["recent"], case["keep"]
        kept, best = s["kept"].long(), s["scores_out"].double()
        out = {n: s[n].double() for n in ("k", "v")}
        for r, n in enumerate(lens):
            for h in range(hkv):
                p = torch.arange(n, device="cuda")
                if n > keep:
                    middle = s["scores"][r, h, first:n - recent]
                    order = torch.sort(-middle.double(), stable=True).indices[:keep - first - recent] + first
                    p = torch.cat([p[:first], order.sort().values, p[n - recent:]])
                new = torch.arange(p.numel(), device="cuda")
                kept[r, h, :p.numel()], best[r, h, :p.numel()] = p, s["scores"][r, h, p].double()
                to, at = s["table_out"][r, new // page].long(), s["table"][r, p // page].long()
                for t in ("k", "v"):
                    out[t][to, new % page, h] = s[t][at, p % page, h].double()
        return dict(out, kept=kept, scores_out=best, lens_out=torch.tensor([min(n, keep) for n in lens], device="cuda"))
    grp = case["grp"]
    o = torch.zeros(case["T"], hkv * grp, D, dtype=torch.float64, device="cuda")
    scores = s["scores"].double()
    for r in range(case["R"]):
        n, t0, t1 = lens[r], begin[r], begin[r + 1]
        where = s["table"][r].long()
        keys, vals = (s[x][where].reshape(-1, hkv, D)[:n + t1 - t0] for x in ("k", "v"))
        scores[r, :, n:n + t1 - t0] = 0
        for t in range(t0, t1):
            bits = int(s["anc"][t]) & 0xFFFFFFFF
            at = torch.tensor([u - t0 + n for u in range(t0, t1) if bits >> u & 1], dtype=torch.long, device="cuda")
            at = torch.cat([torch.arange(n, device="cuda"), at])
            for h in range(hkv):
                z = s["q"][t, h * grp:(h + 1) * grp].double() @ keys[at, h].double().t() / math.sqrt(D)
                e = torch.exp(z - z.max(1, keepdim=True).values)
                e /= e.sum(1, keepdim=True)
                o[t, h * grp:(h + 1) * grp] = e @ vals[at, h].double()
                scores[r, h, at] += e.sum(0)
    return {"o": o, "scores": scores}
