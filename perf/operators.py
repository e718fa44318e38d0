"""The operators of a linear-attention mixer layer in front of the MoE block, as they are measured.

Three operators that run one after another in such a layer:

  norm    residual addition and root-mean-square norm of a token's row, kept in the row's type or
          quantised to e4m3 with one float32 scale per token
              s = x + residual,  y = s * rsqrt(mean(s^2) + eps) * weight
              scale = max|y| / 448,  code = e4m3(y / scale)            (0 for a row of zeros)
  matmul  matrix product of e4m3 codes with a scale per token and a scale per output channel
              out[t][n] = x_scale[t] * w_scale[n] * sum_k x[t][k] * w[n][k]
  scan    linear attention with one decay per value head, S the head's state [d_v][d_k]
              S <- decay * S + v_t k_t^T,  o_t = S q_t
          over whole prompts (dense or packed ragged sequences) and single tokens of many sequences
"""
import math

import torch

own = False

E4M3_MAX = 448.0
CHUNK = 64


def _norm(name, rows, d, dtype, kind, residual):
    return {"name": name, "op": "norm", "rows": rows, "d": d, "dtype": dtype, "out": kind, "residual": residual}


def _matmul(name, T, N, K):
    return {"name": name, "op": "matmul", "T": T, "N": N, "K": K}


def _scan(name, lens, hk, hv, dk, dv, packed):
    return {"name": name, "op": "scan", "lens": lens, "hk": hk, "hv": hv, "dk": dk, "dv": dv, "packed": packed}


def listed():
    return [
        # the norm before the first projection of one decoded token: pure latency
        _norm("norm_token", 1, 2048, "bf16", "e4m3", True),
        # float32 rows of an odd width, no residual stream, kept in float32 (a final norm)
        _norm("norm_odd_f32", 777, 1001, "f32", "same", False),
        # the norm of a large prefill batch, 16K tokens of the block's width
        _norm("norm_prefill", 16384, 2048, "bf16", "e4m3", True),
        # the fused q, k, v projection (16 key heads, 32 value heads of 128) of one token
        _matmul("matmul_token", 1, 8192, 2048),
        # the output projection of 16 sequences decoded together
        _matmul("matmul_batch16", 16, 2048, 4096),
        # a short prompt and an output width that fills no tile
        _matmul("matmul_ragged", 301, 2500, 2048),
        # the fused q, k, v projection of a 16K-token prefill
        _matmul("matmul_prefill", 16384, 8192, 2048),
        # one token of one sequence: the state passes through once
        _scan("scan_token", "1", 16, 32, 128, 128, False),
        # one token of each of 64 sequences, bound by their states
        _scan("scan_batch64", ",".join(["1"] * 64), 16, 32, 128, 128, False),
        # a 4K-token prompt from a kept state
        _scan("scan_prompt", "4096", 16, 32, 128, 128, False),
        # packed prompts of a serving batch: empty, single-token, odd and long ones
        _scan("scan_ragged", "1,700,0,2049,37,1311,64,300,999", 16, 32, 128, 128, True),
        # a long document in one call
        _scan("scan_long", "32768", 16, 32, 128, 128, False),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["norm", "matmul", "scan"])
    if op == "norm":
        while True:
            rows, d = _log(rng, 1, 65536), _log(rng, 64, 8192)
            d = d if rng.random() < 0.5 else max(64, d // 64 * 64)
            dtype = rng.choice(["bf16", "bf16", "f32"])
            if rows * d * (2 if dtype == "f32" else 1) <= 16384 * 2048:
                break
        c = _norm("", rows, d, dtype, rng.choice(["e4m3", "e4m3", "same"]), rng.random() < 0.6)
    elif op == "matmul":
        while True:
            T, N, K = _log(rng, 1, 16384), _log(rng, 16, 16384), 16 * _log(rng, 4, 512)
            if T * N * K <= 16384 * 8192 * 2048 and N * K <= 32 << 20 and T * N <= 128 << 20 and T * K <= 32 << 20:
                break
        c = _matmul("", T, N, K)
    else:
        hk = rng.choice([1, 2, 4, 8, 16])
        hv = hk * rng.choice([1, 2, 4])
        dk, dv = rng.choice([64, 128, 128]), rng.choice([64, 128, 128, 80])
        while True:
            kind = rng.choice(["tokens", "tokens", "dense", "packed", "packed"])
            if kind == "tokens":  # single tokens of many sequences
                lens = [1] * _log(rng, 1, 192)
            elif kind == "dense":  # one prompt, or a few of one length
                lens = [_log(rng, 2, 8192)] * rng.randint(1, 3)
            else:  # packed prompts, some empty or of one token
                lens = [rng.choice([0, 1, _log(rng, 2, 3000), _log(rng, 2, 3000)]) for _ in range(rng.randint(2, 8))]
                lens.append(rng.randint(1, 200))
            if len(lens) * hv <= 4096 and sum(lens) * hv <= 32768 * 32:
                break
        packed = kind == "packed"
        c = _scan("", ",".join(map(str, lens)), hk, hv, dk, dv, packed)
    del c["name"]
    return c


def _type(case):
    return torch.bfloat16 if case["dtype"] == "bf16" else torch.float32


def _lens(case):
    return [int(x) for x in case["lens"].split(",")]


def _quantise_rows(w):
    """e4m3 codes and a float32 scale per row, by the norm's rule."""
    w = w.float()
    scale = w.abs().amax(dim=-1) / E4M3_MAX
    return (w / scale[:, None]).to(torch.float8_e4m3fn), scale


def prepare(case, seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(int(seed))

    def normal(*shape, std=1.0):
        return torch.randn(shape, generator=g, device="cuda", dtype=torch.float32) * std

    s = {"case": dict(case)}
    if case["op"] == "norm":
        t = _type(case)
        rows, d = case["rows"], case["d"]
        # the residual stream's rows differ in size, and a few channels are large
        size = torch.exp(normal(rows, 1, std=0.5))
        channel = torch.exp(normal(d, std=0.3))
        s["x"] = normal(rows, d).to(t)
        s["residual"] = (normal(rows, d) * size * channel).to(t) if case["residual"] else None
        s["weight"] = (1.0 + normal(d, std=0.1)).to(t)
        s["eps"] = 1e-6
        return s
    if case["op"] == "matmul":
        T, N, K = case["T"], case["N"], case["K"]
        s["x"], s["x_scale"] = _quantise_rows(normal(T, K) * torch.exp(normal(K, std=0.3)))
        s["w"], s["w_scale"] = _quantise_rows(normal(N, K, std=K ** -0.5))
        return s
    lens = _lens(case)
    n, N = len(lens), sum(lens)
    hk, hv, dk, dv = case["hk"], case["hv"], case["dk"], case["dv"]

    def unit(*shape):
        x = normal(*shape)
        return x / x.norm(dim=-1, keepdim=True)

    shape = (N,) if case["packed"] else (n, lens[0])
    s["q"] = (unit(*shape, hk, dk) * dk ** -0.5).to(torch.bfloat16)
    s["k"] = unit(*shape, hk, dk).to(torch.bfloat16)
    s["v"] = normal(*shape, hv, dv).to(torch.bfloat16)
    # decays from a memory of a dozen tokens to one of a few thousand
    s["decay"] = 1.0 - torch.exp(torch.linspace(math.log(1 / 12), math.log(1 / 3000), hv, device="cuda") + normal(hv, std=0.1))
    s["state"] = normal(n, hv, dv, dk, std=0.1)
    s["offsets"] = None
    s["longest"] = max(lens)
    if case["packed"]:
        ends = torch.tensor([0] + lens, dtype=torch.int64).cumsum(0)
        s["offsets"] = ends.to(dtype=torch.int32, device="cuda")
    return s


def _plain_norm(s):
    case, t = s["case"], s["x"].dtype
    h = s["x"].float()
    if case["residual"]:
        h = h + s["residual"].float()
    y = h * torch.rsqrt((h * h).mean(dim=-1, keepdim=True) + s["eps"]) * s["weight"].float()
    got = {"sum": h.to(t)} if case["residual"] else {}
    if case["out"] == "same":
        got["out"] = y.to(t)
        return got
    scale = y.abs().amax(dim=-1) / E4M3_MAX
    got["codes"] = torch.where(scale[:, None] == 0, 0.0, y / scale[:, None]).to(torch.float8_e4m3fn)
    got["scales"] = scale
    return got


def _plain_matmul(s):
    y = torch.matmul(s["x"].float(), s["w"].float().t())
    return (y * s["x_scale"][:, None] * s["w_scale"][None, :]).to(torch.bfloat16)


def _plain_scan(s):
    """Chunks of tokens: decayed scores inside a chunk, the state before it across chunks."""
    q, k, v, lam, S0 = s["q"].float(), s["k"].float(), s["v"].float(), s["decay"], s["state"]
    n, hv = S0.shape[0], S0.shape[1]
    L = s["longest"]
    C = min(CHUNK, L)
    nc = -(-L // C)
    at = torch.arange(nc * C, device=q.device)
    if s["offsets"] is None:
        length = torch.full((n,), L, device=q.device)
        first = torch.arange(n, device=q.device) * L
    else:
        first = s["offsets"][:-1].long()
        length = s["offsets"][1:].long() - first
    q, k, v = (x.reshape(-1, *x.shape[-2:]) for x in (q, k, v))
    inside = at[None, :] < length[:, None]  # [n][nc * C]
    row = torch.where(inside, first[:, None] + at[None, :], 0)

    def chunks(x):  # [n][nc][heads of v][C][width], zero past a sequence's end
        x = torch.where(inside[..., None, None], x[row], 0.0)
        x = x.repeat_interleave(hv // x.shape[2], dim=2)
        return x.reshape(n, nc, C, hv, -1).transpose(2, 3)

    qc, kc, vc = chunks(q), chunks(k), chunks(v)
    i = torch.arange(C, device=q.device)
    gap = i[:, None] - i[None, :]
    lam_ = lam[:, None, None]
    inner = torch.where(gap >= 0, lam_ ** gap.clamp(min=0), 0.0)  # [hv][C][C]
    o = torch.matmul(torch.matmul(qc, kc.transpose(-1, -2)) * inner, vc)
    # the state before chunk c: what each earlier chunk left, and the initial one, decayed
    left = torch.matmul((vc * lam_ ** (C - 1 - i)[None, :, None]).transpose(-1, -2), kc)
    c = torch.arange(nc, device=q.device)
    gap = c[:, None] - 1 - c[None, :]
    across = torch.where(gap >= 0, (lam_ ** C) ** gap.clamp(min=0), 0.0)  # [hv][nc][nc]
    before = torch.einsum("hcd,ndhvk->nchvk", across, left)
    before = before + (lam[None, :] ** (C * c)[:, None])[None, :, :, None, None] * S0[:, None]
    o = o + lam_ ** (i + 1)[None, :, None] * torch.matmul(qc, before.transpose(-1, -2))
    o = o.transpose(2, 3).reshape(n, nc * C, hv, -1)[inside].to(torch.bfloat16)
    # the final state: what is in the last chunk reaches the sequence's end only
    last = ((length - 1).clamp(min=0)) // C
    rest = (length - last * C)[:, None, None] - 1 - i[None, None, :]  # [n][1][C]
    w = torch.where(rest >= 0, lam[None, :, None] ** rest.clamp(min=0), 0.0)
    each = torch.arange(n, device=q.device)
    S = torch.matmul((vc[each, last] * w[..., None]).transpose(-1, -2), kc[each, last])
    S = S + (lam[None, :] ** (length - last * C)[:, None])[..., None, None] * before[each, last]
    return {"out": o.reshape(s["v"].shape), "state": S}


def run(state):
    s, op = state, state["case"]["op"]
    if not own:
        return {"norm": _plain_norm, "matmul": _plain_matmul, "scan": _plain_scan}[op](s)
    import sparse_mixture_experts_gemm_gb300 as moe

    if op == "matmul":
        return moe.matmul_fp8(s["x"], s["x_scale"], s["w"], s["w_scale"])
    if op == "scan":
        o, S = moe.gdn_decay_scan(s["q"], s["k"], s["v"], s["decay"], state=s["state"], offsets=s["offsets"])
        return {"out": o, "state": S}
    if s["case"]["out"] == "same":
        out, h = moe.add_rmsnorm(s["x"], s["weight"], residual=s["residual"], eps=s["eps"])
        got = {"out": out}
    else:
        codes, scales, h = moe.add_rmsnorm_fp8(s["x"], s["weight"], residual=s["residual"], eps=s["eps"])
        got = {"codes": codes, "scales": scales}
    if h is not None:
        got["sum"] = h
    return got


def work(case):
    if case["op"] == "norm":
        rows, d, b = case["rows"], case["d"], 2 if case["dtype"] == "bf16" else 4
        n = rows * d
        read = n * b * (2 if case["residual"] else 1) + d * b
        wrote = (n * b if case["residual"] else 0) + (n + 4 * rows if case["out"] == "e4m3" else n * b)
        return {"bytes": read + wrote, "flops": 6 * n}
    if case["op"] == "matmul":
        T, N, K = case["T"], case["N"], case["K"]
        return {"bytes": T * K + N * K + 4 * (T + N) + 2 * T * N, "flops": 2 * T * N * K}
    lens = _lens(case)
    n, N = len(lens), sum(lens)
    hk, hv, dk, dv = case["hk"], case["hv"], case["dk"], case["dv"]
    # the recurrence itself: decay and write (3 operations an element), read (2)
    return {"bytes": N * (2 * 2 * hk * dk + 2 * 2 * hv * dv) + 2 * 4 * n * hv * dv * dk + 4 * hv,
            "flops": 5 * N * hv * dv * dk}


def exact(case, seed):
    s = prepare(case, seed)
    if case["op"] == "norm":
        x = s["x"].double()
        if case["residual"]:
            x = x + s["residual"].double()
        got = {"sum": x} if case["residual"] else {}
        rms = torch.sqrt(x.pow(2).sum(1) / case["d"] + s["eps"])
        y = x / rms[:, None] * s["weight"].double()
        if case["out"] == "same":
            return {**got, "out": y}
        top = y.abs().max(1).values
        return {**got, "codes": y * (E4M3_MAX / top)[:, None], "scales": top / E4M3_MAX}
    if case["op"] == "matmul":
        w = s["w"].double() * s["w_scale"].double()[:, None]
        return (s["x"].double() * s["x_scale"].double()[:, None]) @ w.t()
    # token by token, all sequences side by side
    lens, hv = _lens(case), case["hv"]
    first = [sum(lens[:i]) for i in range(len(lens))]
    q, k, v = (s[x].reshape(-1, *s[x].shape[-2:]).double() for x in "qkv")
    q, k = (x.repeat_interleave(hv // case["hk"], dim=1) for x in (q, k))
    S, lam = s["state"].double(), s["decay"].double()[:, None, None]
    o = torch.zeros_like(v)
    order = sorted(range(len(lens)), key=lambda i: -lens[i])
    back = torch.tensor(sorted(range(len(order)), key=lambda i: order[i]), device=S.device)
    S = S[torch.tensor(order, device=S.device)].clone()
    starts = torch.tensor([first[i] for i in order], device=S.device)
    live = len(order)
    for t in range(max(lens)):
        while live and lens[order[live - 1]] <= t:
            live -= 1
        at = starts[:live] + t
        now = S[:live].mul_(lam)
        now.addcmul_(v[at][..., :, None], k[at][..., None, :])
        o[at] = torch.matmul(now, q[at][..., None])[..., 0]
    return {"out": o.reshape(s["v"].shape), "state": S[back]}
