"""Further operators of a decode step, as measured work.

Three operators that a program calls around the quantized products and the
paged cache: the norm of queries and keys for each head with the position
rotation (qk_norm_rope_run), attention for a batch whose requests share a long
prefix (kv_prefix_attention_run), and sampling the next tokens from the output
head's logits (sample_run).

A case is a dict of plain values; prepare() makes its inputs on the GPU from a
seed; run() makes one pass through the operator, in its plain form (elementary
torch operations in 32 bits, in 64 for angles and for what decides a token) or,
where `own` is true, through the framework's call.  exact() computes the same
outputs in 64 bits, written apart from both.

Byte order of a cache block (one page and head, tokens t, dimensions d):
 keys    [t/16][d/16][t%16][d%16]
 values  [t/32][d/32][(t%16)/4][d%16][(d/16)%2][(t/16)%2][t%4]
"""
import math

import numpy as np
import torch

own = False

DEV = "cuda"


# ------------------------------------------------------------------ the cases
def listed():
    return [
        # one decode step of one stream, heads of the 4096-wide model: latency
        dict(name="rope decode", op="rope", M=1, Hkv=8, G=4, D=128, Dr=128, x="bf16", norm=True, pairs="halves", axes=1, far=8192),
        # a 32-row verification tile from the fp32 product, text among images: positions on three axes
        dict(name="rope axes", op="rope", M=32, Hkv=8, G=4, D=128, Dr=128, x="f32", norm=True, pairs="halves", axes=3, far=131072),
        # a long prompt, every dimension rotated
        dict(name="rope prompt", op="rope", M=5003, Hkv=8, G=4, D=128, Dr=128, x="bf16", norm=True, pairs="halves", axes=1, far=131072),
        # wide heads of which a quarter is rotated, neighbours as pairs, no norm
        dict(name="rope partial", op="rope", M=1021, Hkv=4, G=8, D=256, Dr=64, x="bf16", norm=False, pairs="neighbours", axes=1, far=1 << 20),
        # one stream's next token with the usual filters
        dict(name="sample one", op="sample", M=1, V=151936, x="bf16", temp=0.7, k=50, p=0.9, minp=0.0),
        # a 16-row verification tile, fp32 logits, nucleus only
        dict(name="sample nucleus", op="sample", M=16, V=151936, x="f32", temp=0.8, k=0, p=0.95, minp=0.0),
        # a serving batch whose requests each have their own settings
        dict(name="sample batch", op="sample", M=192, V=151936, x="bf16", temp=-1.0, k=0, p=1.0, minp=0.0),
        # four streams behind one system prompt: the cache's stream
        dict(name="prefix few", op="prefix", R=4, T=1, P=8192, len_max=501, page=64, Hkv=8, G=4, D=128, fmt="int8", tree=False),
        # a serving batch behind a long document, one token each
        dict(name="prefix batch", op="prefix", R=48, T=1, P=32768, len_max=2000, page=64, Hkv=8, G=4, D=128, fmt="int8", tree=False),
        # the same kind of batch verifying draft trees: many rows a head
        dict(name="prefix verify", op="prefix", R=16, T=16, P=20011, len_max=700, page=64, Hkv=8, G=4, D=128, fmt="int8", tree=True),
        # wide heads, a very long document, e4m3 codes
        dict(name="prefix long", op="prefix", R=8, T=1, P=131072, len_max=300, page=128, Hkv=4, G=8, D=256, fmt="e4m3", tree=False),
        # many streams just after a short common opening: latency
        dict(name="prefix short", op="prefix", R=32, T=1, P=333, len_max=64, page=32, Hkv=8, G=4, D=128, fmt="int8", tree=False),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["rope", "sample", "sample", "prefix", "prefix"])
    if op == "rope":
        D = rng.choice([64, 80, 96, 128, 128, 256])
        Dr = rng.choice([D, D, D, 32, 64])
        Hkv, G = _log(rng, 1, 16), rng.choice([1, 2, 3, 4, 5, 8])
        M = max(1, min(_log(rng, 1, 8192), 5003 * 5120 // ((Hkv + Hkv * G) * D)))
        return dict(op=op, M=M, Hkv=Hkv, G=G, D=D, Dr=Dr, x=rng.choice(["bf16", "f32"]), norm=rng.random() < 0.75,
                    pairs=rng.choice(["halves", "neighbours"]), axes=rng.choice([1, 1, 2, 3]), far=_log(rng, 100, 1 << 24))
    if op == "sample":
        V = _log(rng, 1000, 262144)
        M = max(1, min(_log(rng, 1, 256), 192 * 151936 // V))
        if rng.random() < 0.4:
            return dict(op=op, M=M, V=V, x=rng.choice(["bf16", "f32"]), temp=-1.0, k=0, p=1.0, minp=0.0)
        return dict(op=op, M=M, V=V, x=rng.choice(["bf16", "f32"]), temp=rng.choice([0.0, 0.5, 0.8, 1.0, 1.3]),
                    k=rng.choice([0, 0, 1, 20, 50, 200]), p=rng.choice([1.0, 1.0, 0.5, 0.9, 0.95]), minp=rng.choice([0.0, 0.0, 0.02, 0.1]))
    D = rng.choice([64, 128, 128, 256])
    page = rng.choice([32, 64, 128, 256])
    R, Hkv, G = _log(rng, 1, 96), _log(rng, 1, 8), rng.choice([1, 2, 3, 4, 5, 7, 8])
    T = 1 if rng.random() < 0.5 else _log(rng, 2, 32)
    most = 16 * 16 * 32 * 20011 * 128 // (R * T * Hkv * G * D)
    P = max(1, min(_log(rng, 1, 131072), 131072 * 1024 // (Hkv * D), most))
    ln = max(T, min(_log(rng, 1, 4000), 48 * 2000 * 1024 // (R * Hkv * D), most // 4))
    return dict(op=op, R=R, T=T, P=P, len_max=ln, page=page, Hkv=Hkv, G=G, D=D, fmt=rng.choice(["int8", "e4m3"]),
                tree=T > 1 and rng.random() < 0.5)


# ------------------------------------------------------------------ inputs
def _rng(seed, item=0):
    return np.random.default_rng([int(seed), item])


def _gen(seed):
    g = torch.Generator(device=DEV)
    g.manual_seed(int(seed))
    return g


def _dt(name):
    return {"bf16": torch.bfloat16, "f32": torch.float32}[name]


def _i32(a):
    return torch.from_numpy(np.ascontiguousarray(a, dtype=np.int32)).to(DEV)


def _f32(a):
    return torch.from_numpy(np.ascontiguousarray(a, dtype=np.float32)).to(DEV)


def _codes(shape, fmt, g):
    """Codes as a quantizer leaves them: int8 near a normal's, e4m3 likewise."""
    n = math.prod(shape)
    out = torch.empty(n, dtype=torch.uint8, device=DEV)
    step = 1 << 27
    for a in range(0, n, step):
        b = min(n, a + step)
        z = torch.randn(b - a, device=DEV, generator=g)
        if fmt == "int8":
            out[a:b] = z.mul_(40).round_().clamp_(-127, 127).to(torch.int8).view(torch.uint8)
        else:
            out[a:b] = z.mul_(140).clamp_(-448, 448).to(torch.float8_e4m3fn).view(torch.uint8)
        del z
    return out.view(torch.int8 if fmt == "int8" else torch.float8_e4m3fn).view(shape)


def _prepare_rope(s, case, seed, g):
    M, Hkv, D, Dr = (case[k] for k in ("M", "Hkv", "D", "Dr"))
    Hq = Hkv * case["G"]
    # the joint projection's output, its values behind the queries and keys
    qkv = torch.randn(M, Hq + 2 * Hkv, D, device=DEV, generator=g)
    qkv[:, :, :: max(1, D // 3)] *= 6
    s["qkv"] = qkv.to(_dt(case["x"]))
    s["q"], s["k"] = s["qkv"][:, :Hq], s["qkv"][:, Hq:Hq + Hkv]
    s["qw"], s["kw"] = ((1 + 0.2 * torch.randn(D, device=DEV, generator=g)).to(torch.bfloat16) if case["norm"] else None
                        for _ in range(2))
    s["inv_freq"] = _f32(10000.0 ** (-np.arange(Dr // 2) * 2.0 / Dr))
    r = _rng(seed)
    if case["axes"] == 1:
        start = int(r.integers(0, max(1, case["far"] - M)))
        s["positions"] = _i32(start + np.arange(M))
        s["axis"] = None
    else:
        s["positions"] = _i32(r.integers(0, case["far"], (case["axes"], M)))
        s["axis"] = torch.from_numpy((np.arange(Dr // 2) * case["axes"] // (Dr // 2)).astype(np.uint8)).to(DEV)
    s["q_out"] = torch.empty(M, Hq, D, dtype=torch.bfloat16, device=DEV)
    s["k_out"] = torch.empty(M, Hkv, D, dtype=torch.bfloat16, device=DEV)


def _prepare_sample(s, case, seed, g):
    M, V = case["M"], case["V"]
    # an output head's logits: a broad body, and a few tokens that the context
    # points at, more or less clearly from row to row
    x = 2.2 * torch.randn(M, V, device=DEV, generator=g)
    n = min(60, V)
    at = torch.randint(0, V, (M, n), device=DEV, generator=g)
    lift = torch.empty(M, n, device=DEV).exponential_(1.0, generator=g) * 3 + 5
    x.scatter_add_(1, at, lift * (0.5 + torch.rand(M, 1, device=DEV, generator=g)))
    s["logits"] = x.to(_dt(case["x"]))
    r = _rng(seed)
    if case["temp"] < 0:
        s["temperature"] = _f32(r.choice([0.0, 0.5, 0.7, 1.0, 1.2], M))
        s["top_k"] = _i32(r.choice([0, 0, 1, 20, 50, 1000], M))
        s["top_p"] = _f32(r.choice([1.0, 1.0, 0.5, 0.9, 0.95], M))
        s["min_p"] = _f32(r.choice([0.0, 0.0, 0.0, 0.02, 0.1], M))
    else:
        s["temperature"] = _f32(np.full(M, case["temp"])) if case["temp"] != 1 else None
        s["top_k"] = _i32(np.full(M, case["k"])) if case["k"] else None
        s["top_p"] = _f32(np.full(M, case["p"])) if case["p"] < 1 else None
        s["min_p"] = _f32(np.full(M, case["minp"])) if case["minp"] else None
    s["u"] = torch.rand(M, device=DEV, generator=g)
    s["tokens"] = torch.empty(M, dtype=torch.int32, device=DEV)
    s["logprobs"] = torch.empty(M, device=DEV)


def _prepare_prefix(s, case, seed, g):
    R, T, P, page, Hkv, G, D = (case[k] for k in ("R", "T", "P", "page", "Hkv", "G", "D"))
    r = _rng(case["len_max"], R)  # the same lengths for every seed, in another order
    ln = np.exp(r.uniform(0, math.log(case["len_max"] + 1), R)).astype(np.int64)
    n = np.full(R, T)
    n[1:] = np.where(r.random(R - 1) < 0.7, T, r.integers(1, T + 1, R - 1))
    ln = np.clip(ln, n, max(case["len_max"], T))
    ln[-1], n[-1] = max(case["len_max"], T), T
    if R > 8:
        n[1::16] = 0  # idle requests
    r = _rng(seed)
    order = r.permutation(R)
    ln, n = ln[order], n[order]
    nb, pb = -(-ln // page), -(-P // page)
    pages = int(nb.sum()) + pb + 3
    perm = r.permutation(pages)
    cols = max(1, int(nb.max()))
    table = np.full((R, cols), -1, np.int32)
    table[np.arange(cols)[None, :] < nb[:, None]] = perm[: nb.sum()]
    q_start = np.concatenate([[0], np.cumsum(n)])
    M = int(q_start[-1])
    s.update(lens=_i32(ln), q_start=_i32(q_start), table=_i32(table), M=M, cols=cols, max_q=T,
             prefix_table=_i32(perm[nb.sum(): nb.sum() + pb]), prefix_len=_i32([P]))
    s["q"] = torch.randn(M, Hkv * G, D, device=DEV, generator=g).to(torch.bfloat16)
    for name in ("k", "v"):
        s[name] = _codes((pages, Hkv, page, D), case["fmt"], g)
        s[name + "_scales"] = (0.5 + torch.rand(pages, Hkv, device=DEV, generator=g)) * (0.025 if case["fmt"] == "int8" else 0.007)
    if case["tree"]:  # random trees: each draft token's parent is an earlier one, or the context
        masks = []
        for m in n:
            seen = []
            for j in range(m):
                p = int(r.integers(-1, j)) if j else -1
                seen.append((seen[p] if p >= 0 else 0) | (1 << j))
            masks += seen
        s["tree_mask"] = _i32(np.array(masks, dtype=np.uint32).view(np.int32))
    s["out"] = torch.empty(M, Hkv * G, D, dtype=torch.bfloat16, device=DEV)


def prepare(case, seed):
    s = dict(case)
    {"rope": _prepare_rope, "sample": _prepare_sample, "prefix": _prepare_prefix}[case["op"]](s, case, seed, _gen(seed))
    return s


# ------------------------------------------------------------------ one pass
def run(s):
    if own:
        return _run_own(s)
    return {"rope": _rope, "sample": _sample, "prefix": _prefix}[s["op"]](s)


def _run_own(s):
    import quantized_weight_decode_dequant_amd as qg
    if s["op"] == "rope":
        return qg.qk_norm_rope_run(s["q"], s["k"], s["positions"], s["inv_freq"], q_weight=s["qw"], k_weight=s["kw"], eps=1e-6,
                                   axis=s["axis"], interleaved=s["pairs"] == "neighbours", q_out=s["q_out"], k_out=s["k_out"])
    if s["op"] == "sample":
        return qg.sample_run(s["logits"], s["u"], temperature=s["temperature"], top_k=s["top_k"], top_p=s["top_p"],
                             min_p=s["min_p"], tokens=s["tokens"], logprobs=s["logprobs"])
    if "cache" not in s:  # the handle a program makes once for a layer
        s["cache"] = qg.KVCache(s["k"], s["v"], s["k_scales"], s["v_scales"])
    return qg.kv_prefix_attention_run(s["cache"], s["q"], s["q_start"], s["lens"], s["table"], s["prefix_table"], s["prefix_len"],
                                      s["max_q"], tree_mask=s.get("tree_mask"), out=s["out"])


def _rope(s):
    D, Dr = s["D"], s["Dr"]
    pos = s["positions"].view(s["axes"], -1)
    at = pos[0][:, None] if s["axis"] is None else pos[s["axis"].long()].t()
    angle = at.double() * s["inv_freq"].double()
    c, sn = angle.cos().float()[:, None], angle.sin().float()[:, None]
    out = []
    for x, w in ((s["q"], s["qw"]), (s["k"], s["kw"])):
        x = x.float()
        if w is not None:
            x = x * torch.rsqrt((x * x).mean(2, keepdim=True) + 1e-6) * w.float()
        if s["pairs"] == "halves":
            a, b = x[..., : Dr // 2], x[..., Dr // 2: Dr]
            x = torch.cat([a * c - b * sn, b * c + a * sn, x[..., Dr:]], 2)
        else:
            a, b = x[..., 0:Dr:2], x[..., 1:Dr:2]
            x = torch.cat([torch.stack([a * c - b * sn, b * c + a * sn], 3).flatten(2), x[..., Dr:]], 2)
        out.append(x.to(torch.bfloat16))
    return out


def _sample(s):
    M, V = s["M"], s["V"]
    ones = torch.ones(M, 1, dtype=torch.float64, device=DEV)
    T = s["temperature"].double()[:, None] if s["temperature"] is not None else ones
    k = s["top_k"].long()[:, None] if s["top_k"] is not None else torch.zeros(M, 1, dtype=torch.int64, device=DEV)
    p = s["top_p"].double()[:, None] if s["top_p"] is not None else ones
    minp = s["min_p"].double()[:, None] if s["min_p"] is not None else 0 * ones
    k = torch.where(T == 0, 1, torch.where((k <= 0) | (k > V), V, k))  # temperature 0: the largest
    # the largest first, equal ones in their order; 64 bits, as a sum decides which token it is
    x, order = torch.sort(s["logits"].double(), dim=1, descending=True, stable=True)
    w = torch.exp((x - x[:, :1]) / torch.where(T == 0, 1.0, T))
    rank = torch.arange(V, device=DEV)[None]
    w = torch.where(rank < k, w, 0.0)
    S = w.sum(1, keepdim=True)
    keep = (rank == 0) | ((p >= 1) | (w.cumsum(1) - w < p * S)) & (w >= minp)
    w = torch.where(keep, w, 0.0)
    w = torch.zeros_like(w).scatter_(1, order, w)  # the tokens' order again
    c = w.cumsum(1)
    at = torch.searchsorted(c, s["u"].double()[:, None] * c[:, -1:], right=True)
    at = torch.minimum(at, torch.searchsorted(c, c[:, -1:].contiguous()))  # not past the last one kept
    return [at.view(M).int(), torch.log(w.gather(1, at) / c[:, -1:]).view(M).float()]


def _rows_k(c, D):
    """Key blocks [..., page, D] in the cache's byte order -> row-major."""
    lead, page = c.shape[:-2], c.shape[-2]
    n = len(lead)
    c = c.reshape(*lead, page // 16, D // 16, 16, 16)
    return c.permute(*range(n), n, n + 2, n + 1, n + 3).reshape(*lead, page, D)


def _rows_v(c, D):
    """Value blocks in the cache's byte order -> row-major."""
    lead, page = c.shape[:-2], c.shape[-2]
    n = len(lead)
    c = c.reshape(*lead, page // 32, D // 32, 4, 16, 2, 2, 4)
    return c.permute(*range(n), n, n + 5, n + 2, n + 6, n + 1, n + 4, n + 3).reshape(*lead, page, D)


def _tokens(s, name, ids):
    """The pages `ids` [n, blocks] of one side: values [n, Hkv, tokens, D] and their scales [n, Hkv, tokens]."""
    page, Hkv, D = s["page"], s["Hkv"], s["D"]
    n, L = ids.shape[0], ids.shape[1] * page
    rows = (_rows_k if name == "k" else _rows_v)(s[name].view(torch.uint8)[ids], D).view(s[name].dtype)
    return (rows.transpose(1, 2).reshape(n, Hkv, L, D).float(),
            s[name + "_scales"][ids].transpose(1, 2).repeat_interleave(page, 2, output_size=L))


def _prefix(s):
    R, Hkv, G, D, M, T, P = (s[k] for k in ("R", "Hkv", "G", "D", "M", "max_q", "P"))
    L = s["cols"] * s["page"]
    q0, ln = s["q_start"][:-1].long(), s["lens"].long()
    n = s["q_start"][1:].long() - q0
    j = torch.arange(T, device=DEV)
    row = (q0[:, None] + j).clamp(max=M - 1)
    q = s["q"].float() / math.sqrt(D)
    # the prefix, for all rows of a head at once
    ids = s["prefix_table"].long()[None]
    K, ks = _tokens(s, "k", ids)
    S1 = (q.view(M, Hkv, G, D).transpose(0, 1).reshape(Hkv, M * G, D) @ K[0].transpose(1, 2)) * ks[0][:, None, :]
    S1 = torch.where(torch.arange(K.shape[2], device=DEV) < P, S1, -math.inf)
    m1 = S1.amax(2, keepdim=True)
    # each request's own tokens
    ids = s["table"].clamp(min=0).long()
    K, ks = _tokens(s, "k", ids)
    S2 = (q[row].view(R, T, Hkv, G, D).transpose(1, 2).reshape(R, Hkv, T * G, D) @ K.transpose(2, 3)) * ks[:, :, None, :]
    base = (ln - n)[:, None, None]
    t = torch.arange(L, device=DEV)
    see = (t <= base + j[None, :, None]) & (t < ln[:, None, None])
    if s["tree"]:
        bits = s["tree_mask"].long()[row][:, :, None] >> (t - base).clamp(0, 31)
        see = (t < base) | (((bits & 1) > 0) & (t < ln[:, None, None]))
    S2 = torch.where(see[:, None, :, None, :].expand(R, 1, T, G, L).reshape(R, 1, T * G, L), S2, -math.inf)
    # one maximum for a row's two parts
    m1r = m1.view(Hkv, M, G).transpose(0, 1)[row].transpose(1, 2).reshape(R, Hkv, T * G, 1)
    m2 = torch.maximum(S2.amax(3, keepdim=True), m1r)
    to = torch.where(j < n[:, None], q0[:, None] + j, M).view(-1)  # padded rows go to a spare last one

    def back(x):  # [R, Hkv, T * G, ...] -> [M, Hkv, G, ...]
        x = x.reshape(R, Hkv, T, G, -1).transpose(1, 2).reshape(R * T, Hkv, G, -1)
        return torch.zeros(M + 1, *x.shape[1:], device=DEV).index_copy(0, to, x)[:M]

    m = back(m2).transpose(0, 1).reshape(Hkv, M * G, 1)
    P1 = torch.exp(S1 - m)
    del S1
    V, vs = _tokens(s, "v", s["prefix_table"].long()[None])
    l1, o1 = P1.sum(2), (P1 * vs[0][:, None, :]) @ V[0]
    P2 = torch.exp(S2 - m2)
    V, vs = _tokens(s, "v", ids)
    l2, o2 = back(P2.sum(3)), back((P2 * vs[:, :, None, :]) @ V)
    l = l1.view(Hkv, M, G).transpose(0, 1)[..., None] + l2
    o = o1.view(Hkv, M, G, D).transpose(0, 1) + o2
    return (o / l).reshape(M, Hkv * G, D).to(torch.bfloat16)


# ------------------------------------------------------------------ what a pass needs
def _prefix_rows(case):
    """Query tokens of a call, as _prepare_prefix makes them, and cached tokens of the requests."""
    R, T = case["R"], case["T"]
    r = _rng(case["len_max"], R)
    ln = np.exp(r.uniform(0, math.log(case["len_max"] + 1), R)).astype(np.int64)
    n = np.full(R, T)
    n[1:] = np.where(r.random(R - 1) < 0.7, T, r.integers(1, T + 1, R - 1))
    ln = np.clip(ln, n, max(case["len_max"], T))
    ln[-1], n[-1] = max(case["len_max"], T), T
    if R > 8:
        n[1::16] = 0
    return n, np.where(n > 0, ln, 0)


def work(case):
    if case["op"] == "rope":
        n = case["M"] * case["Hkv"] * (1 + case["G"]) * case["D"]
        size = {"bf16": 2, "f32": 4}[case["x"]]
        return {"bytes": n * (size + 2) + 4 * case["M"] * case["axes"] + 2 * case["Dr"] + 4 * case["D"] * case["norm"],
                "flops": n * (4 * case["norm"] + 3 * case["Dr"] / case["D"])}
    if case["op"] == "sample":
        n = case["M"] * case["V"]
        return {"bytes": n * {"bf16": 2, "f32": 4}[case["x"]] + 28 * case["M"], "flops": 2 * n}
    n, ln = _prefix_rows(case)
    H, G, D, P = case["Hkv"], case["G"], case["D"], case["P"]
    return {"bytes": int((P + ln.sum()) * H * D * 2 + n.sum() * H * G * D * 4),
            "flops": int(4 * H * G * D * (n.sum() * P + (n * ln).sum()))}


# ------------------------------------------------------------------ the definition, in 64 bits
def exact(case, seed):
    s = prepare(case, seed)
    return {"rope": _rope64, "sample": _sample64, "prefix": _prefix64}[case["op"]](s)


def _rope64(s):
    D, half = s["D"], s["Dr"] // 2
    pos = s["positions"].double().reshape(s["axes"], s["M"])
    freq = s["inv_freq"].double()
    turn = torch.empty(s["M"], half, dtype=torch.complex128, device=DEV)
    for i in range(half):
        a = pos[0 if s["axis"] is None else int(s["axis"][i])] * freq[i]
        turn[:, i] = torch.polar(torch.ones_like(a), a)
    out = []
    for x, w in ((s["q"], s["qw"]), (s["k"], s["kw"])):
        y = x.double().clone()
        if w is not None:
            y *= (y.square().sum(2, keepdim=True) / D + 1e-6) ** -0.5
            y *= w.double()
        a = torch.arange(half, device=DEV) * (1 if s["pairs"] == "halves" else 2)
        b = a + (half if s["pairs"] == "halves" else 1)
        z = torch.complex(y[:, :, a], y[:, :, b]) * turn[:, None]
        y[:, :, a], y[:, :, b] = z.real, z.imag
        out.append(y)
    return out


def _sample64(s):
    V = s["V"]
    host = {n: (s[n].tolist() if s[n] is not None else [off] * s["M"])
            for n, off in (("temperature", 1.0), ("top_k", 0), ("top_p", 1.0), ("min_p", 0.0), ("u", 0.0))}
    logp = []
    for m in range(s["M"]):
        T, k, p, minp, u = (host[n][m] for n in ("temperature", "top_k", "top_p", "min_p", "u"))
        # distinct values, the largest first, and how many tokens have each
        vals, which, count = torch.unique(s["logits"][m].double(), return_inverse=True, return_counts=True)
        vals, count, which = vals.flip(0), count.flip(0), len(vals) - 1 - which
        if T == 0:
            k, T = 1, 1.0
        k = V if k <= 0 else min(k, V)
        kept = torch.minimum((k - (count.cumsum(0) - count)).clamp(min=0), count)
        w = torch.exp((vals - vals[0]) / T)
        if p < 1:
            mass = w * kept
            room = p * mass.sum() - (mass.cumsum(0) - mass)
            kept = torch.minimum(kept, torch.ceil(room / w).clamp(min=0).nan_to_num(0, 0, 0).long())
        kept = torch.where(w >= minp, kept, 0)
        kept[0] = max(int(kept[0]), 1)
        # a value's tokens in their order: the first kept[value] of them
        take = kept[which] == count[which]
        part = torch.nonzero((kept > 0) & (kept < count)).view(-1).tolist()
        for v in part:
            take[torch.nonzero(which == v).view(-1)[: int(kept[v])]] = True
        ids = torch.nonzero(take).view(-1)
        c = w[which[ids]].cumsum(0)
        i = min(int((c <= u * c[-1]).sum()), len(ids) - 1)
        logp.append(float(vals[which[ids[i]]] - vals[0]) / T - math.log(float(c[-1])))
    return [None, torch.tensor(logp, dtype=torch.float64, device=DEV)]


def _place(page, D, value):
    """Byte offset of (token, dimension) in a block."""
    t, d = np.arange(page)[:, None], np.arange(D)[None, :]
    if not value:
        off = (t // 16) * 16 * D + (d // 16) * 256 + (t % 16) * 16 + d % 16
    else:
        off = (t // 32) * 32 * D + (d // 32) * 1024 + (t % 16 // 4) * 256 + (d % 16) * 16 + (d // 16 % 2) * 8 + (t // 16 % 2) * 4 + t % 4
    return torch.from_numpy(off.reshape(-1)).to(DEV)


def _prefix64(s):
    page, Hkv, G, D, M = (s[k] for k in ("page", "Hkv", "G", "D", "M"))
    start, lens = s["q_start"].tolist(), s["lens"].tolist()
    place = {"k": _place(page, D, False), "v": _place(page, D, True)}

    def cached(name, ids, h, n):
        codes = s[name].view(torch.uint8)[ids, h].view(len(ids), -1)[:, place[name]].view(s[name].dtype).double()
        return (codes.view(-1, page, D) * s[name + "_scales"][ids, h].double()[:, None, None]).view(-1, D)[:n]

    out = torch.zeros(M, Hkv * G, D, dtype=torch.float64, device=DEV)
    for h in range(Hkv):
        K0, V0 = (cached(x, s["prefix_table"].long(), h, s["P"]) for x in ("k", "v"))
        for r in range(s["R"]):
            a, b, n = start[r], start[r + 1], lens[r]
            T = b - a
            if T == 0:
                continue
            ids = s["table"][r, : -(-n // page)].long()
            K, V = torch.cat([K0, cached("k", ids, h, n)]), torch.cat([V0, cached("v", ids, h, n)])
            new = torch.arange(-s["P"], n, device=DEV)[None, :] - (n - T)
            if s["tree"]:
                seen = torch.where(new < 0, 1, (s["tree_mask"][a:b].long()[:, None] >> new.clamp(min=0)) & 1).bool()
            else:
                seen = new <= torch.arange(T, device=DEV)[:, None]
            w = torch.mm(s["q"][a:b, h * G:(h + 1) * G].double().reshape(T * G, D), K.t().contiguous()) * D ** -0.5
            w = w.masked_fill(~seen.repeat_interleave(G, 0), -math.inf)
            out[a:b, h * G:(h + 1) * G] = torch.mm(torch.softmax(w, 1), V).view(T, G, D)
    return out
