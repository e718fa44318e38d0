"""The operators of a full-attention layer, as they are measured.

They run one after another in the attention layers that a hybrid model has between its linear ones:

  rope     root-mean-square norm of every query and key head with the position rotation in the same pass
               y = x * rsqrt(mean(x^2) + eps) * weight                     over a head's D columns
               the first R columns in pairs (i, i + R / 2), a = position * inv_freq[i]:
               out[i] = y[i] cos a - y[i + R/2] sin a,  out[i + R/2] = y[i + R/2] cos a + y[i] sin a
  prefill  causal attention of prompts, several query heads on one key/value head, packed sequences; the
           queries of a sequence are the last of its keys
               o_i = sum_j softmax_j(scale * q_i . k_j) v_j                over keys j <= i + (keys - queries)
  cache    keys and values quantised to 4 bits as they are written into pages of 64 tokens, and read back
               per 64 columns: bias = bf16(min), scale = bf16((max - min) / 15),
               code = round((x - bias) / scale) in 0 .. 15,  value = bf16(scale * code + bias)
  decode   attention of one new token per sequence over such a cache
               o = sum_t softmax_t(scale * q . k_t) v_t                    over the tokens in the cache

A cache is two tensors: codes uint8 [pages][2][heads][64][D / 2] (keys, then values; the even column in the
low half of a byte) and affine bf16 [pages][2][heads][64][D / 64][2] (scale, bias).  A table of page numbers
per sequence says where its tokens are.
"""
import math

import torch

own = False

PAGE, GROUP = 64, 64
EPS = 1e-6


def _rope(name, tokens, hq, hk, d, rot):
    return {"name": name, "op": "rope", "tokens": tokens, "hq": hq, "hk": hk, "d": d, "rot": rot}


def _prefill(name, q_lens, k_lens, hq, hk, d):
    return {"name": name, "op": "prefill", "q_lens": q_lens, "k_lens": k_lens, "hq": hq, "hk": hk, "d": d}


def _cache(name, starts, lens, hk, d):
    return {"name": name, "op": "cache", "starts": starts, "lens": lens, "hk": hk, "d": d}


def _decode(name, lens, hq, hk, d):
    return {"name": name, "op": "decode", "lens": lens, "hq": hq, "hk": hk, "d": d}


def listed():
    ragged = "1,700,0,2049,37,1311,64,300,999"
    # 64 sequences decoded together, from a few tokens of context to 8K
    contexts = [16 + (i * 1237 + 401) % 8177 for i in range(64)]
    return [
        # one decoded token: pure latency
        _rope("rope_token", 1, 16, 2, 256, 64),
        # a 16K-token prefill batch
        _rope("rope_prefill", 16384, 16, 2, 256, 64),
        # a prompt of one line
        _prefill("prefill_line", "17", "17", 16, 2, 256),
        # packed prompts of a serving batch: empty, single-token, odd and long ones
        _prefill("prefill_ragged", ragged, ragged, 16, 2, 256),
        # a 4K-token prompt
        _prefill("prefill_prompt", "4096", "4096", 16, 2, 256),
        # heads of 128 with less sharing, a batch of equal prompts
        _prefill("prefill_heads128", "2048,2048", "2048,2048", 32, 8, 128),
        # the last 8K-token piece of a 32K-token document
        _prefill("prefill_piece", "8192", "32768", 16, 2, 256),
        # one new token of each of 64 sequences
        _cache("cache_tokens", ",".join(map(str, contexts)), ",".join(["1"] * 64), 2, 256),
        # a 16K-token prompt written and read back
        _cache("cache_prompt", "0", "16384", 2, 256),
        # a token of one sequence behind a 4K-token prompt
        _decode("decode_one", "4097", 16, 2, 256),
        # a serving batch
        _decode("decode_batch64", ",".join(map(str, contexts)), 16, 2, 256),
        # a token behind a long document
        _decode("decode_long", "131072", 16, 2, 256),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["rope", "prefill", "prefill", "cache", "decode", "decode"])
    d = rng.choice([128, 256, 256])
    hk = rng.choice([1, 2, 2, 4, 8])
    hq = hk * rng.choice([1, 2, 3, 4, 8, 8])
    most = {c["name"]: c for c in listed()}
    if op == "rope":
        while True:
            tokens = _log(rng, 1, 65536)
            if tokens * (hq + hk) * d <= 16384 * 18 * 256:
                break
        c = _rope("", tokens, hq, hk, d, rng.choice([32, 64, 96, 128, d]))
    elif op == "prefill":
        top = work(most["prefill_piece"])["flops"]
        while True:
            kind = rng.choice(["one", "packed", "packed", "behind"])
            if kind == "one":  # one prompt
                ql = kl = [_log(rng, 1, 16384)]
            elif kind == "packed":  # prompts of a batch, some empty or of one token
                ql = [rng.choice([0, 1, _log(rng, 2, 3000), _log(rng, 2, 3000)]) for _ in range(rng.randint(2, 10))]
                ql.append(rng.randint(1, 200))
                kl = ql
            else:  # pieces behind tokens that are in the cache already
                ql = [_log(rng, 1, 4096) for _ in range(rng.randint(1, 4))]
                kl = [n + rng.choice([0, _log(rng, 1, 16384)]) for n in ql]
            c = _prefill("", ",".join(map(str, ql)), ",".join(map(str, kl)), hq, hk, d)
            if work(c)["flops"] <= top and max(sum(ql), 1) * hq * d <= 1 << 27:
                break
    elif op == "cache":
        while True:
            n = rng.choice([1, rng.randint(2, 8), _log(rng, 8, 128)])
            lens = [1] * n if n > 8 else [rng.choice([0, 1, _log(rng, 2, 8192)]) for _ in range(n)]
            starts = [rng.choice([0, _log(rng, 1, 16384)]) for _ in lens]
            if 0 < sum(lens) * hk * d <= 16384 * 512 and sum(lens) + sum(starts) <= 1 << 18:
                break
        c = _cache("", ",".join(map(str, starts)), ",".join(map(str, lens)), hk, d)
    else:
        top = work(most["decode_batch64"])["bytes"]
        while True:
            n = _log(rng, 1, 128)
            longest = _log(rng, 1, 131072)
            lens = [rng.choice([longest, rng.randint(0, longest), rng.randint(0, longest)]) for _ in range(n)]
            c = _decode("", ",".join(map(str, lens)), hq, hk, d)
            if work(c)["bytes"] <= top and n * max(lens) * hk * d <= 64 * 8192 * 512 and max(lens) > 0:
                break
    del c["name"]
    return c


def _ints(text):
    return [int(x) for x in text.split(",")]


def _ends(lens):
    return torch.tensor([0] + lens, dtype=torch.int64).cumsum(0).to(dtype=torch.int32, device="cuda")


def _quantise(x):
    """codes (one per byte), scale and bias of x [..., D] in groups of 64."""
    g = x.float().unflatten(-1, (-1, GROUP))
    lo, hi = g.amin(-1), g.amax(-1)
    bias = lo.to(torch.bfloat16)
    scale = ((hi - lo) / 15).to(torch.bfloat16)
    s, b = scale.float()[..., None], bias.float()[..., None]
    code = torch.where(s == 0, 0.0, torch.round((g - b) / s)).clamp(0, 15)
    return code.flatten(-2).to(torch.uint8), scale, bias


def _pack(x):
    """x [..., D] as a cache holds it: two codes per byte, scale next to bias."""
    code, scale, bias = _quantise(x)
    return code[..., 0::2] | code[..., 1::2] << 4, torch.stack([scale, bias], -1)


def _unpack(codes, affine):
    """float32 values of a cache's rows [..., D / 2], [..., D / 64, 2]"""
    c = torch.stack([codes & 15, codes >> 4], -1).flatten(-2).float()
    a = affine.float()
    return (c.unflatten(-1, (-1, GROUP)) * a[..., 0:1] + a[..., 1:2]).flatten(-2)


def prepare(case, seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(int(seed))

    def normal(*shape, std=1.0):
        return torch.randn(shape, generator=g, device="cuda", dtype=torch.float32) * std

    op, hk, d = case["op"], case["hk"], case["d"]
    s = {"case": dict(case)}
    bf16 = torch.bfloat16
    # keys and values: some columns larger than others, as trained norms leave them
    column = torch.exp(normal(d, std=0.3))
    if op == "rope":
        N, hq, rot = case["tokens"], case["hq"], case["rot"]
        # slices of one fused projection, the sizes of tokens apart
        qkv = (normal(N, hq + 2 * hk, d) * torch.exp(normal(N, 1, 1, std=0.5))).to(bf16)
        s["q"], s["k"] = qkv[:, :hq], qkv[:, hq:hq + hk]
        s["q_weight"], s["k_weight"] = ((1 + normal(d, std=0.1)).to(bf16) for _ in range(2))
        first = int(torch.randint(0, 120000, (1,), generator=g, device="cuda"))
        s["positions"] = torch.arange(first, first + N, dtype=torch.int32, device="cuda")
        s["inv_freq"] = 1e7 ** (-torch.arange(0, rot, 2, dtype=torch.float64, device="cuda") / rot)
        return s
    if op == "prefill":
        ql, kl, hq = _ints(case["q_lens"]), _ints(case["k_lens"]), case["hq"]
        s["q"] = (normal(sum(ql), hq, d) * 1.5).to(bf16)
        s["k"] = (normal(sum(kl), hk, d) * column).to(bf16)
        s["v"] = normal(sum(kl), hk, d).to(bf16)
        s["offsets"], s["k_offsets"] = _ends(ql), _ends(kl) if ql != kl else None
        return s
    lens = _ints(case["lens"])
    n = len(lens)
    reach = [a + b for a, b in zip(_ints(case["starts"]), lens)] if op == "cache" else lens
    width = max(1, -(-max(reach) // PAGE))
    need = [-(-x // PAGE) for x in reach]
    P = sum(need) + 3
    order = torch.randperm(P, generator=g, device="cuda").to(torch.int32)
    table = torch.zeros(n, width, dtype=torch.int32, device="cuda")
    at = 0
    for i, x in enumerate(need):
        table[i, :x] = order[at:at + x]
        at += x
    s["pages"] = table
    if op == "cache":
        s["codes"] = torch.zeros(P, 2, hk, PAGE, d // 2, dtype=torch.uint8, device="cuda")
        s["affine"] = torch.zeros(P, 2, hk, PAGE, d // GROUP, 2, dtype=bf16, device="cuda")
        s["k"] = (normal(sum(lens), hk, d) * column).to(bf16)
        s["v"] = normal(sum(lens), hk, d).to(bf16)
        s["starts"] = torch.tensor(_ints(case["starts"]), dtype=torch.int32, device="cuda")
        s["offsets"] = _ends(lens)
        return s
    values = normal(P, 2, hk, PAGE, d)
    values[:, 0] *= column
    s["codes"], s["affine"] = _pack(values)
    s["q"] = (normal(n, case["hq"], d) * 1.5).to(bf16)
    s["lengths"] = torch.tensor(lens, dtype=torch.int32, device="cuda")
    return s


def _plain_rope(s):
    rot = s["case"]["rot"]
    half = rot // 2
    angle = s["positions"].double()[:, None] * s["inv_freq"]
    cos, sin = angle.cos().float()[:, None], angle.sin().float()[:, None]
    got = []
    for x, w in ((s["q"], s["q_weight"]), (s["k"], s["k_weight"])):
        y = x.float()
        y = y * torch.rsqrt((y * y).mean(-1, keepdim=True) + EPS) * w.float()
        a, b = y[..., :half], y[..., half:rot]
        got.append(torch.cat([a * cos - b * sin, b * cos + a * sin, y[..., rot:]], -1).to(torch.bfloat16))
    return {"q": got[0], "k": got[1]}


def _attend(q, k, v, first, kind):
    """Queries q [Lq][Hq][D], query i seeing keys up to first + i, in blocks that bound the scores' memory."""
    Lq, hq, d = q.shape
    Lk, hk = k.shape[:2]
    kt, vt = k.to(kind).permute(1, 2, 0), v.to(kind).transpose(0, 1)
    o = torch.empty(Lq, hq, d, dtype=kind, device=q.device)
    step = max(1, min(Lq, (1 << 28) // max(1, hq * Lk)))
    for a in range(0, Lq, step):
        b = min(Lq, a + step)
        seen = min(Lk, first + b)
        x = q[a:b].to(kind).unflatten(1, (hk, -1)).permute(1, 2, 0, 3)  # [hk][group][block][D]
        x = torch.matmul(x, kt[:, None, :, :seen]) * d ** -0.5
        i = torch.arange(a, b, device=q.device)
        x = torch.where(torch.arange(seen, device=q.device)[None, :] <= first + i[:, None], x, -math.inf)
        x = torch.exp(x - x.amax(-1, keepdim=True))
        x = torch.matmul(x, vt[:, None, :seen]) / x.sum(-1, keepdim=True)
        o[a:b] = x.permute(2, 0, 1, 3).flatten(1, 2)
    return o


def _prefill_as(s, kind):
    ql, kl = _ints(s["case"]["q_lens"]), _ints(s["case"]["k_lens"])
    parts, a, b = [], 0, 0
    for x, y in zip(ql, kl):
        if x:
            parts.append(_attend(s["q"][a:a + x], s["k"][b:b + y], s["v"][b:b + y], y - x, kind))
        a, b = a + x, b + y
    return torch.cat(parts) if parts else s["q"].to(kind)


def _slots(s):
    """Page and place in it of every token of a cache call."""
    lens = _ints(s["case"]["lens"])
    N = sum(lens)
    row = torch.arange(N, device="cuda")
    seq = torch.searchsorted(s["offsets"][1:].long(), row, right=True)
    at = row - s["offsets"].long()[seq] + s["starts"].long()[seq]
    return s["pages"].long()[seq, at // PAGE], at % PAGE


def _plain_cache(s):
    page, place = _slots(s)
    for i, x in enumerate((s["k"], s["v"])):
        codes, affine = _pack(x)
        s["codes"][page, i, :, place] = codes
        s["affine"][page, i, :, place] = affine
    got = [_unpack(s["codes"][page, i, :, place], s["affine"][page, i, :, place]).to(torch.bfloat16) for i in (0, 1)]
    return {"k": got[0], "v": got[1]}


def _plain_decode(s):
    case, n = s["case"], s["q"].shape[0]
    hk, d = case["hk"], case["d"]
    scale = d ** -0.5
    L = s["pages"].shape[1] * PAGE
    q = s["q"].float().unflatten(1, (hk, -1))
    o = torch.empty_like(q)
    step = max(1, (1 << 27) // (L * hk * d))  # sequences at a time
    for a in range(0, n, step):
        pages = s["pages"][a:a + step].long()
        k, v = (_unpack(s["codes"][pages, i], s["affine"][pages, i]).transpose(1, 2).flatten(2, 3) for i in (0, 1))
        inside = torch.arange(L, device=q.device)[None, :] < s["lengths"][a:a + step, None]
        v = torch.where(inside[:, None, :, None], v, 0.0)
        x = torch.matmul(q[a:a + step], k.transpose(-1, -2)) * scale
        x = torch.where(inside[:, None, None], x, -math.inf)
        top = x.amax(-1, keepdim=True)
        x = torch.exp(x - torch.where(top == -math.inf, 0.0, top))
        total = x.sum(-1, keepdim=True)
        o[a:a + step] = torch.matmul(x, v) / torch.where(total == 0, 1.0, total)
    return o.flatten(1, 2).to(torch.bfloat16)


def run(state):
    s, op = state, state["case"]["op"]
    if not own:
        if op == "prefill":
            return _prefill_as(s, torch.float32).to(torch.bfloat16)
        return {"rope": _plain_rope, "cache": _plain_cache, "decode": _plain_decode}[op](s)
    import sparse_mixture_experts_gemm_gb300 as moe

    if op == "rope":
        q, k = moe.qk_norm_rope(s["q"], s["k"], s["q_weight"], s["k_weight"], s["positions"], s["inv_freq"], eps=EPS)
        return {"q": q, "k": k}
    if op == "prefill":
        return moe.attention_prefill(s["q"], s["k"], s["v"], offsets=s["offsets"], k_offsets=s["k_offsets"])
    cache = (s["codes"], s["affine"])
    if op == "cache":
        moe.kv_cache_write(cache, s["k"], s["v"], s["pages"], s["starts"], offsets=s["offsets"])
        k, v = moe.kv_cache_read(cache, s["pages"], s["offsets"], s["k"].shape[0], starts=s["starts"])
        return {"k": k, "v": v}
    return moe.attention_decode(s["q"], cache, s["pages"], s["lengths"])


def work(case):
    op, hk, d = case["op"], case["hk"], case["d"]
    if op == "rope":
        n = case["tokens"] * (case["hq"] + hk) * d
        return {"bytes": 4 * n + 4 * d + case["tokens"] * 4 + 4 * case["rot"], "flops": 6 * n}
    if op == "prefill":
        ql, kl, hq = _ints(case["q_lens"]), _ints(case["k_lens"]), case["hq"]
        pairs = sum(x * (y - x) + x * (x + 1) // 2 for x, y in zip(ql, kl))
        return {"bytes": 4 * sum(ql) * hq * d + 4 * sum(kl) * hk * d, "flops": 4 * pairs * hq * d}
    row = d // 2 + d // 16  # bytes of a head's keys or values of a token in the cache
    N = sum(_ints(case["lens"]))
    if op == "cache":
        return {"bytes": 2 * N * hk * 2 * (2 * d + row), "flops": 2 * N * hk * d * 8}
    n, hq = len(_ints(case["lens"])), case["hq"]
    return {"bytes": 2 * N * hk * row + 4 * n * hq * d, "flops": 4 * N * hq * d}


def exact(case, seed):
    s = prepare(case, seed)
    op, d = case["op"], case["d"]
    if op == "rope":
        half = case["rot"] // 2
        turn = torch.polar(torch.ones((), dtype=torch.float64, device="cuda"),
                           s["positions"].double()[:, None] * s["inv_freq"])[:, None]
        got = {}
        for name in "qk":
            x = s[name].double()
            x = x / torch.sqrt(x.pow(2).sum(-1, keepdim=True) / d + EPS) * s[name + "_weight"].double()
            z = torch.complex(x[..., :half], x[..., half:2 * half]) * turn
            got[name] = torch.cat([z.real, z.imag, x[..., 2 * half:]], -1)
        return got
    if op == "prefill":
        # every query head by itself, against the keys that its block of rows sees
        ql, kl, group = _ints(case["q_lens"]), _ints(case["k_lens"]), case["hq"] // case["hk"]
        o = torch.zeros(s["q"].shape, dtype=torch.float64, device="cuda")
        a0 = b0 = 0
        for x, y in zip(ql, kl):
            for a in range(0, x, 512):
                b = min(x, a + 512)
                seen = y - x + b
                late = torch.triu(torch.ones(b - a, seen, dtype=torch.bool, device="cuda"), y - x + a + 1)
                for h in range(case["hq"]):
                    k, v = (s[t][b0:b0 + seen, h // group].double() for t in "kv")
                    z = (s["q"][a0 + a:a0 + b, h].double() @ k.t()) / math.sqrt(d)
                    o[a0 + a:a0 + b, h] = torch.softmax(z.masked_fill(late, -math.inf), -1) @ v
            a0, b0 = a0 + x, b0 + y
        return o
    if op == "cache":
        got = {}
        for name in "kv":
            x = s[name].double().unflatten(-1, (-1, GROUP))
            low = x.amin(-1, keepdim=True)
            scale = ((x.amax(-1, keepdim=True) - low) / 15).to(torch.bfloat16).double()
            low = low.to(torch.bfloat16).double()
            code = torch.round((x - low) / torch.where(scale == 0, 1.0, scale)).clamp(0, 15)
            got[name] = (low + scale * code).flatten(-2)
        return got
    o = torch.zeros(s["q"].shape, dtype=torch.float64, device="cuda")
    group = case["hq"] // case["hk"]
    for i, length in enumerate(_ints(case["lens"])):
        if length == 0:
            continue
        table = s["pages"][i, :-(-length // PAGE)].long()
        for h in range(case["hk"]):
            kv = []
            for which in (0, 1):
                c = s["codes"][table, which, h].flatten(0, 1)[:length]
                a = s["affine"][table, which, h].flatten(0, 1)[:length].double()
                x = torch.empty(length, d, dtype=torch.float64, device="cuda")
                x[:, 0::2], x[:, 1::2] = (c % 16).double(), (c // 16).double()
                x = x.unflatten(-1, (-1, GROUP)) * a[..., :1] + a[..., 1:]
                kv.append(x.flatten(-2))
            z = s["q"][i, h * group:(h + 1) * group].double() @ kv[0].t() / math.sqrt(d)
            o[i, h * group:(h + 1) * group] = torch.softmax(z, -1) @ kv[1]
    return o
