"""Cases and reference forms of the 4-bit and attention operators.

Three kinds of work, each in a plain form (elementary torch operations in 32
bits, rounded once at the end) and, with ``own`` true, as the calls that a
user makes of the package:

  quantize  fp16/fp32 rows -> 4-bit rows with group scales, and back
  matmul    y = W x over 4-bit rows, 1..32 tokens
  ffn       the sparse FFN over a list of active neurons, 4-bit rows
  tree      append the drafted tokens' keys and values to a paged cache, then
            attention of the drafted tokens over it

A 4-bit row of k weights is kp/2 bytes of codes (kp = k rounded up to a
multiple of 128) followed by its fp16 group scales, zero padded to
``row_bytes``.  Weight i is (code - 8) * scale[i // group].  In each block of
128 weights (16 words of 32 bits), word 4t+j holds weights 32j+8t .. 32j+8t+7;
weight 2p+h of a word is the nibble at bit 16h+4p.  Weights past k have code 8.
"""
import math

import torch

own = False


# ------------------------------------------------------------------ cases --
def listed():
    return [
        # a whole fp16 projection of the 7B shape brought to 4 bits at load time
        dict(name="quantize 7B up f16 g128", kind="quantize", m=11008, k=4096, group=128, dtype="f16"),
        # an fp32 layer of the tiny shape with a ragged row length and the finest groups
        dict(name="quantize ragged f32 g32", kind="quantize", m=1376, k=1000, group=32, dtype="f32"),
        # one token through a square projection: the call whose latency counts
        dict(name="matmul 7B square b1", kind="matmul", m=4096, k=4096, B=1, group=128, dtype="f16"),
        # one token through the widest dense product of the 70B shape
        dict(name="matmul 70B up b1", kind="matmul", m=28672, k=8192, B=1, group=128, dtype="f16"),
        # the same for the largest batch, finer groups
        dict(name="matmul 70B up b32 g64", kind="matmul", m=28672, k=8192, B=32, group=64, dtype="f16"),
        # fp32 activations, odd row count, a row length that ends inside a block
        dict(name="matmul ragged f32 b3 g32", kind="matmul", m=5003, k=2760, B=3, group=32, dtype="f32"),
        # one token of the tiny fp32 layer: launch latency
        dict(name="ffn tiny f32 b1", kind="ffn", act="reglu", d=512, n=1376, active=140, B=1, group=32, dtype="f32"),
        # one token of the 70B shape over its predicted list
        dict(name="ffn 70B reglu b1", kind="ffn", act="reglu", d=8192, n=28672, active=3440, B=1, group=128, dtype="f16"),
        # sixteen tokens of the OPT shape over the union of their lists
        dict(name="ffn OPT relu b16", kind="ffn", act="relu", d=12288, n=49152, active=13000, B=16, group=128,
             dtype="f16"),
        # one new token after a short prompt, heads of their own
        dict(name="tree short b1", kind="tree", R=1, T=1, L=333, hkv=32, grp=1, D=128, page=16, ragged=False),
        # requests of very different lengths, a few drafted tokens each, 64-wide heads
        dict(name="tree ragged r8", kind="tree", R=8, T=32, L=9001, hkv=8, grp=16, D=64, page=16, ragged=True),
        # sixteen drafted tokens of one long conversation, grouped heads
        dict(name="tree long t16", kind="tree", R=1, T=16, L=65500, hkv=8, grp=8, D=128, page=64, ragged=False),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    kind = rng.choice(["quantize", "matmul", "matmul", "ffn", "ffn", "tree", "tree"])
    group = rng.choice([32, 64, 128])
    dtype = rng.choice(["f16", "f16", "f32"])
    if kind == "quantize":
        k = 8 * _log(rng, 8, 1536)
        m = min(_log(rng, 64, 20000), 11008 * 4096 // k)
        return dict(kind=kind, m=m, k=k, group=group, dtype=dtype)
    if kind == "matmul":
        k = 8 * _log(rng, 8, 3584)
        B = rng.choice([1, 1, 2, rng.randint(3, 8), rng.randint(9, 32)])
        m = max(1, min(_log(rng, 64, 49152), 28672 * 8192 // k))
        return dict(kind=kind, m=m, k=k, B=B, group=group, dtype=dtype)
    if kind == "ffn":
        d = 8 * _log(rng, 16, 1536)
        n = max(8, min(_log(rng, 400, 49152), 28672 * 8192 // d))
        B = rng.choice([1, 1, 2, rng.randint(3, 8), rng.randint(9, 32)])
        return dict(kind=kind, act=rng.choice(["relu", "reglu"]), d=d, n=n,
                    active=max(1, int(n * rng.uniform(0.02, 0.35))), B=B, group=group, dtype=dtype)
    R = rng.choice([1, 1, 2, 5, 16, 32])
    T = rng.randint(R, 32)
    hkv = rng.choice([1, 2, 8, 32])
    grp = rng.choice([1, 1, 4, 7, 8, 16]) if hkv < 32 else 1
    L = _log(rng, 1, 60000 // (R * max(1, hkv // 8)) + 2)
    return dict(kind=kind, R=R, T=T, L=L, hkv=hkv, grp=grp, D=rng.choice([64, 80, 128]),
                page=rng.choice([16, 20, 64, 256]), ragged=rng.random() < 0.5)


def _bits(group):
    return 0.5 + 2.0 / group


def work(case):
    if case["kind"] == "quantize":
        e = 2 if case["dtype"] == "f16" else 4
        mk = case["m"] * case["k"]
        return {"bytes": mk * (2 * e + 2 * _bits(case["group"])), "flops": 4 * mk}
    if case["kind"] == "matmul":
        e = 2 if case["dtype"] == "f16" else 4
        m, k, B = case["m"], case["k"], case["B"]
        return {"bytes": m * k * _bits(case["group"]) + B * (k * e + m * 4), "flops": 2 * m * k * B}
    if case["kind"] == "ffn":
        e = 2 if case["dtype"] == "f16" else 4
        w = case["active"] * (3 if case["act"] == "reglu" else 2) * case["d"]
        B, d = case["B"], case["d"]
        return {"bytes": w * _bits(case["group"]) + B * d * (e + 4) + case["active"] * 8, "flops": 2 * w * B}
    lens, begin = _requests(case)
    T, hkv, grp, D = case["T"], case["hkv"], case["grp"], case["D"]
    seen = sum(lens[r] + begin[r + 1] - begin[r] for r in range(case["R"]))
    pairs = sum((begin[r + 1] - begin[r]) * (lens[r] + begin[r + 1] - begin[r]) for r in range(case["R"]))
    return {"bytes": 4 * D * hkv * (seen + 2 * T) + 4 * D * hkv * grp * T, "flops": 4 * D * hkv * grp * pairs}


# ----------------------------------------------------------------- inputs --
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
    c = c.view(m, kp // 128, 4, 4, 4, 2)                                  # block, j, t, p, h
    at = torch.tensor([[0, 16], [4, 20], [8, 24], [12, 28]], device=w.device, dtype=torch.int32)
    words = (c << at).sum((-1, -2), dtype=torch.int32)                    # nibbles do not overlap: a sum is an or
    codes = words.transpose(-1, -2).contiguous().view(torch.uint8).view(m, kp // 2)
    out = torch.zeros(m, _row_bytes(k, group), dtype=torch.uint8, device=w.device)
    out[:, :kp // 2] = codes
    out[:, kp // 2:kp // 2 + 2 * (kp // group)] = s.contiguous().view(torch.uint8).view(m, -1)
    return out


def _packed_normal(m, k, std, group, gen):
    """Normal weights, packed a few thousand rows at a time."""
    step = max(1, (1 << 26) // k)
    return torch.cat([_pack(torch.randn(min(step, m - i), k, generator=gen, device="cuda") * std, group)
                      for i in range(0, m, step)])


def _requests(case):
    """Prefix lengths and token ranges of the requests: fixed by the case."""
    R, T, L = case["R"], case["T"], case["L"]
    if case["ragged"]:
        lens = [max(0, L * (r * 7 % R + 1) // R - 1 - r) for r in range(R)]
        if R > 2:
            lens[2] = 0                                                    # a request that has only just begun
    else:
        lens = [max(0, L - r) for r in range(R)]
    begin = [T * r // R for r in range(R + 1)]
    return lens, begin


def prepare(case, seed):
    gen = torch.Generator(device="cuda").manual_seed(seed)

    def normal(*shape):
        return torch.randn(*shape, generator=gen, device="cuda")

    s = dict(case=case, kind=case["kind"])
    if case["kind"] == "tree":
        return _prepare_tree(s, case, gen, normal)
    dt = torch.float16 if case["dtype"] == "f16" else torch.float32
    group = case["group"]
    if case["kind"] == "quantize":
        s["src"] = (normal(case["m"], case["k"]) / math.sqrt(case["k"])).to(dt)
        s["data"] = torch.zeros(case["m"], _row_bytes(case["k"], group), dtype=torch.uint8, device="cuda")
        s["back"] = torch.empty_like(s["src"])
        if own:
            import activation_sparse_ffn_predict_b200 as A
            s["A"], s["mat"] = A, A.W4Matrix(s["data"], case["k"], group)
    elif case["kind"] == "matmul":
        m, k, B = case["m"], case["k"], case["B"]
        s["data"] = _packed_normal(m, k, 1 / math.sqrt(k), group, gen)
        s["x"] = normal(B, k).to(dt)
        s["y"] = torch.empty(B, m, device="cuda")
        if own:
            import activation_sparse_ffn_predict_b200 as A
            s["A"], s["mat"] = A, A.W4Matrix(s["data"], k, group)
            s["ws"] = A.Workspace.for_w4(s["mat"], B)
    else:
        d, n, B, mats = case["d"], case["n"], case["B"], 3 if case["act"] == "reglu" else 2
        rows = [_packed_normal(n, d, 1 / math.sqrt(n if i == mats - 1 else d), group, gen) for i in range(mats)]
        s["data"] = torch.stack(rows, 1).contiguous()                     # [n, mats, row_bytes]
        s["bias"] = normal(n) * 0.5
        s["x"] = normal(B, d).to(dt)
        s["y"] = torch.empty(B, d, device="cuda")
        s["idx"] = torch.zeros(n, dtype=torch.int32, device="cuda")
        act = torch.rand(n, generator=gen, device="cuda").argsort()[:case["active"]].sort().values
        s["idx"][:case["active"]] = act.to(torch.int32)
        s["count"] = torch.full((1,), case["active"], dtype=torch.int32, device="cuda")
        if own:
            import activation_sparse_ffn_predict_b200 as A
            s["A"], s["ffn"] = A, A.W4FFN(case["act"], s["data"], s["bias"], d, group)
            s["ws"] = A.Workspace.for_w4(s["ffn"], B)
    return s


def _prepare_tree(s, case, gen, normal):
    R, T, hkv, grp, D, page = (case[k] for k in ("R", "T", "hkv", "grp", "D", "page"))
    lens, begin = _requests(case)
    need = [-(-(lens[r] + begin[r + 1] - begin[r]) // page) for r in range(R)]
    pages, most = sum(need) + 3, max(need)
    order = torch.rand(pages, generator=gen, device="cuda").argsort().to(torch.int32)
    table = torch.zeros(R, most, dtype=torch.int32, device="cuda")
    at = 0
    for r in range(R):
        table[r, :need[r]] = order[at:at + need[r]]
        at += need[r]
    anc = []
    pick = torch.rand(T, generator=gen, device="cuda").tolist()
    for r in range(R):
        for i in range(begin[r + 1] - begin[r]):
            t = begin[r] + i
            parent = int(pick[t] * (i + 1)) - 1                            # -1: the tree's root follows the prefix
            anc.append((1 << t) | (anc[begin[r] + parent] if parent >= 0 else 0))
    s["anc"] = torch.tensor([a - (1 << 32) if a >> 31 else a for a in anc], dtype=torch.int32, device="cuda")
    s["k"], s["v"] = (normal(pages, page, hkv, D).half() for _ in range(2))
    s["k_new"], s["v_new"] = (normal(T, hkv, D).half() for _ in range(2))
    s["q"] = (normal(T, hkv * grp, D) * 1.5).half()
    s["o"] = torch.empty_like(s["q"])
    s["table"] = table
    s["lens"] = torch.tensor(lens, dtype=torch.int32, device="cuda")
    s["begin"] = torch.tensor(begin, dtype=torch.int32, device="cuda")
    s["most"] = max(lens[r] + begin[r + 1] - begin[r] for r in range(R))
    s["tmax"] = max(begin[r + 1] - begin[r] for r in range(R))
    if own:
        import activation_sparse_ffn_predict_b200 as A
        s["A"], s["cache"] = A, A.KVCache(s["k"], s["v"])
        s["ws"] = A.Workspace.for_attention(s["cache"], hkv * grp, R, T)
    return s


# ------------------------------------------------------------ plain forms --
def _unpack(data, k, group):
    """fp32 rows [..., k] of 4-bit rows [..., row_bytes]."""
    kp = _pad(k)
    lead = data.shape[:-1]
    words = data[..., :kp // 2].contiguous().view(torch.int32).view(*lead, kp // 128, 4, 4).transpose(-1, -2).contiguous()
    at = torch.tensor([0, 16, 4, 20, 8, 24, 12, 28], device=data.device, dtype=torch.int32)
    c = ((words.unsqueeze(-1) >> at) & 15).sub_(8).float().view(*lead, kp // group, group)
    s = data[..., kp // 2:kp // 2 + 2 * (kp // group)].contiguous().view(torch.float16).float()
    return (c * s.unsqueeze(-1)).view(*lead, kp)[..., :k]


def _plain_quantize(s):
    w, group = s["src"].float(), s["case"]["group"]
    m, k = w.shape
    w = torch.nn.functional.pad(w, (0, _pad(k) - k)).view(m, -1, group)
    sf = (w.abs().amax(-1, keepdim=True) / torch.full((), 7.0, device=w.device)).half().float()
    c = torch.where(sf > 0, torch.round(w / sf), torch.zeros_like(w)).clamp_(-8, 7)
    return (c * sf).view(m, -1)[:, :k].to(s["src"].dtype)


def _plain_ffn(s):
    c = s["case"]
    rows = s["idx"][:c["active"]].long()
    w = _unpack(s["data"][rows], c["d"], c["group"])
    x, b = s["x"].float(), s["bias"][rows]
    a = torch.clamp(x @ w[:, 0].t() + b, min=0)
    if c["act"] == "reglu":
        a = a * (x @ w[:, 1].t())
    return a @ w[:, -1]


def _plain_tree(s):
    c = s["case"]
    hkv, grp, D, page, T = c["hkv"], c["grp"], c["D"], c["page"], c["T"]
    lens, begin = s["lens"].long(), s["begin"].long()
    tok = torch.arange(T, device="cuda")
    req = (tok[:, None] >= begin[None, 1:]).sum(1)
    where = lens[req] + tok - begin[req]
    slot = s["table"][req, where // page].long()
    s["k"][slot, where % page] = s["k_new"]
    s["v"][slot, where % page] = s["v_new"]
    p = torch.arange(s["most"], device="cuda")
    j = p[None] - lens[:, None]                                            # [R, P] place among the drafted tokens
    own_t = (begin[1:] - begin[:-1])[:, None]
    drafted = (j >= 0) & (j < own_t)
    bit = torch.where(drafted, begin[:-1, None] + j, torch.zeros_like(j))
    i = torch.arange(s["tmax"], device="cuda")
    rows = torch.where(i[None] < own_t, begin[:-1, None] + i[None], torch.zeros_like(i[None]))  # [R, t]
    sees = (j < 0)[:, None] | (drafted[:, None] & (((s["anc"].long()[rows][:, :, None] >> bit[:, None]) & 1) > 0))
    page_of = s["table"].long()[:, p // page]
    k = s["k"][page_of, p % page].float().permute(0, 2, 3, 1)              # [R, hkv, D, P]
    v = s["v"][page_of, p % page].float().permute(0, 2, 1, 3)              # [R, hkv, P, D]
    q = s["q"].float().view(T, hkv, grp, D)[rows].permute(0, 2, 1, 3, 4).reshape(c["R"], hkv, -1, D)
    z = (q @ k) * (1 / math.sqrt(D))
    z = z.view(c["R"], hkv, -1, grp, s["most"]).masked_fill_(~sees[:, None, :, None], -math.inf)
    top = z.amax(-1, keepdim=True)
    e = torch.exp(z.sub_(torch.where(torch.isinf(top), torch.zeros_like(top), top)))
    total = e.sum(-1, keepdim=True)
    o = (e.view(c["R"], hkv, -1, s["most"]) @ v).view(c["R"], hkv, -1, grp, D)
    o = torch.where(total > 0, o / total, torch.zeros_like(o))
    s["o"][:] = o.permute(0, 2, 1, 3, 4)[req, tok - begin[req]].reshape(T, hkv * grp, D).half()
    return {"o": s["o"], "k": s["k"], "v": s["v"]}


def run(s):
    kind = s["kind"]
    if own:
        A = s["A"]
        if kind == "quantize":
            A.asf_w4_quantize(s["src"], s["mat"])
            A.asf_w4_dequantize(s["mat"], s["back"])
            return s["back"]
        if kind == "matmul":
            A.asf_w4_matmul(s["mat"], s["x"], s["y"], s["ws"])
            return s["y"]
        if kind == "ffn":
            A.asf_w4_sparse_ffn(s["ffn"], s["x"], s["idx"], s["count"], s["y"], s["ws"])
            return s["y"]
        A.asf_kv_append(s["cache"], s["table"], s["lens"], s["begin"], s["k_new"], s["v_new"], s["ws"])
        A.asf_tree_attention(s["cache"], s["table"], s["lens"], s["begin"], s["q"], s["anc"], s["o"], s["ws"])
        return {"o": s["o"], "k": s["k"], "v": s["v"]}
    if kind == "quantize":
        return _plain_quantize(s)
    if kind == "matmul":
        return s["x"].float() @ _unpack(s["data"], s["case"]["k"], s["case"]["group"]).t()
    if kind == "ffn":
        return _plain_ffn(s)
    return _plain_tree(s)


# ------------------------------------------------------- 64-bit definition --
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
    if case["kind"] == "quantize":
        w = s["src"].double()
        out = torch.empty_like(w)
        for a in range(0, case["k"], case["group"]):
            g = w[:, a:a + case["group"]]
            sc = (g.abs().max(1, keepdim=True).values / 7).to(torch.float16).double()
            out[:, a:a + case["group"]] = torch.where(sc > 0, torch.round(g / sc).clamp(-8, 7) * sc, torch.zeros_like(g))
        return out
    if case["kind"] == "matmul":
        step = max(1, (1 << 25) // case["k"])
        x = s["x"].double()
        return torch.cat([x @ _rows64(s["data"][a:a + step], case["k"], case["group"]).t()
                          for a in range(0, case["m"], step)], 1)
    if case["kind"] == "ffn":
        x, y = s["x"].double(), torch.zeros(case["B"], case["d"], dtype=torch.float64, device="cuda")
        step = max(1, (1 << 25) // case["d"])
        listed_rows = s["idx"][:case["active"]].long()
        for a in range(0, case["active"], step):
            at = listed_rows[a:a + step]
            w = [_rows64(s["data"][at, i], case["d"], case["group"]) for i in range(s["data"].shape[1])]
            h = torch.relu(x @ w[0].t() + s["bias"][at].double())
            y += (h * (x @ w[1].t()) if case["act"] == "reglu" else h) @ w[-1]
        return y
    lens, begin = _requests(case)
    hkv, grp, D, page = case["hkv"], case["grp"], case["D"], case["page"]
    o = torch.zeros(case["T"], hkv * grp, D, dtype=torch.float64, device="cuda")
    for r in range(case["R"]):
        n, t0, t1 = lens[r], begin[r], begin[r + 1]
        for i in range(t1 - t0):
            a, b = divmod(n + i, page)
            s["k"][s["table"][r, a], b], s["v"][s["table"][r, a], b] = s["k_new"][t0 + i], s["v_new"][t0 + i]
        where = s["table"][r].long()
        keys = s["k"][where].reshape(-1, hkv, D)[:n + t1 - t0]
        vals = s["v"][where].reshape(-1, hkv, D)[:n + t1 - t0]
        for t in range(t0, t1):
            bits = int(s["anc"][t]) & 0xFFFFFFFF
            at = torch.tensor([u - t0 + n for u in range(t0, t1) if bits >> u & 1], dtype=torch.long, device="cuda")
            at = torch.cat([torch.arange(n, device="cuda"), at])
            for h in range(hkv):
                z = s["q"][t, h * grp:(h + 1) * grp].double() @ keys[at, h].double().t() / math.sqrt(D)
                e = torch.exp(z - z.max(1, keepdim=True).values)
                o[t, h * grp:(h + 1) * grp] = e @ vals[at, h].double() / e.sum(1, keepdim=True)
    return {"o": o, "k": s["k"].double(), "v": s["v"].double()}
