"""The paged key/value cache's operators as measured calls: append, read and attention.

A language model that decodes against cached tokens (one token at a time, a block of tokens
denoised at a time, or a prompt in chunks) appends each chunk's keys and values to pages, attends
the chunk's queries to every cached token, and now and then gathers a range of tokens back into
contiguous K and V, which the block selection and the sparse forward take.

Token j of sequence b lives in page table[b, j // page], slot j % page. kv_len counts the cached
tokens, the chunk's own included; n_new the chunk's tokens (rows past it are padding). An e4m3
cache holds codes with one fp32 scale per token and key/value head.
"""
import math

import torch

own = False


# ---------------------------------------------------------------------------- cases

def _case(name, op, B, H, Hkv, N, d, page, kind, kv, n_lo=None, causal=True, window=0):
    return {"name": name, "op": op, "B": B, "H": H, "Hkv": Hkv, "N": N, "d": d, "page": page, "kind": kind,
            "kv_lo": kv[0], "kv_hi": kv[1], "n_lo": N if n_lo is None else n_lo, "causal": causal, "window": window}


def listed():
    return [
        # attention: the first tokens of one short conversation, where the call's latency counts
        _case("token_short", "attend", 1, 16, 16, 1, 64, 16, "bf16", (437, 437)),
        # a serving batch's decode step: 64 sequences of very different lengths, four query heads a key head
        _case("token_batch", "attend", 64, 32, 8, 1, 128, 64, "bf16", (150, 8100)),
        # few long documents from an 8-bit cache: only a split along the keys fills the GPU
        _case("token_long_e4m3", "attend", 3, 32, 8, 1, 128, 128, "e4m3", (70001, 131072)),
        # a diffusion language model's block of 32 tokens, denoised against its cached prompt, every key kept
        _case("block_bidirectional", "attend", 12, 32, 32, 32, 128, 64, "bf16", (1000, 4500), causal=False),
        # a long prompt's next chunk, causal: bound by the tensor cores
        _case("chunk_causal", "attend", 1, 32, 8, 2048, 128, 64, "bf16", (32768, 32768)),
        # ragged prompts in one padded batch over an 8-bit cache of small pages, five query heads a key head, windowed
        _case("chunk_ragged_e4m3", "attend", 5, 20, 4, 777, 128, 16, "e4m3", (900, 9001), n_lo=190, window=4096),
        # joint text and image tokens against themselves, d = 64, every key kept (the 1024-pixel workload's length)
        _case("chunk_d64", "attend", 2, 24, 24, 1229, 64, 256, "bf16", (4250, 4429), n_lo=1100, causal=False),
        # append: the decode step's one token a sequence into an 8-bit cache
        _case("append_token_e4m3", "append", 64, 32, 8, 1, 128, 64, "e4m3", (150, 8100)),
        # append: prompts of ragged lengths, quantised as they are written
        _case("append_chunk_e4m3", "append", 6, 32, 8, 8192, 128, 16, "e4m3", (8192, 12001), n_lo=2501),
        # append: prompts into bf16 pages
        _case("append_chunk_bf16", "append", 4, 24, 24, 4429, 64, 64, "bf16", (4429, 9000), n_lo=4000),
        # read: long 8-bit caches gathered for the block selection
        _case("read_e4m3", "read", 2, 32, 8, 32768, 128, 64, "e4m3", (30011, 32768)),
        # read: a short bf16 cache of small pages
        _case("read_bf16", "read", 7, 16, 16, 1111, 64, 16, "bf16", (333, 1111)),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["attend", "attend", "attend", "attend", "append", "read"])
    d = rng.choice([64, 128])
    page = rng.choice([16, 32, 64, 128, 256])
    kind = rng.choice(["bf16", "e4m3"])
    Hkv = rng.choice([1, 2, 3, 4, 8, 16, 24])
    G = rng.choice([1, 1, 2, 4, 5, 8])
    if op != "attend":
        B = _log(rng, 1, 48)
        N = _log(rng, 1, 12000)
        N = max(1, min(N, (1 << 28) // (B * Hkv * d)))
        hi = N + rng.randrange(0, 3000)
        lo = max(1, int(hi * rng.uniform(0.3, 1.0)))
        return _unnamed(op, B, Hkv * G, Hkv, N, d, page, kind, lo, hi, max(1, int(N * rng.uniform(0.3, 1.0))), True, 0)
    shape = rng.choice(["token", "few", "chunk"])
    B = _log(rng, 1, 64) if shape != "chunk" else _log(rng, 1, 6)
    N = 1 if shape == "token" else _log(rng, 2, 64) if shape == "few" else _log(rng, 65, 2500)
    hi = max(N, _log(rng, 60, 120000 if shape == "token" else 30000))
    while hi > N and (B * Hkv * hi * d > (1 << 27) or B * Hkv * G * N * hi > (1 << 31)):
        hi = max(N, hi * 2 // 3)
    while B > 1 and (B * Hkv * hi * d > (1 << 27) or B * Hkv * G * N * hi > (1 << 31)):
        B -= 1
    causal = shape == "token" or rng.random() < 0.6
    window = rng.randrange(1, hi + 1) if causal and rng.random() < 0.25 else 0
    lo = max(1, int(hi * rng.uniform(0.1, 1.0)))
    return _unnamed(op, B, Hkv * G, Hkv, N, d, page, kind, lo, hi, max(1, int(N * rng.uniform(0.3, 1.0))), causal, window)


def _unnamed(op, B, H, Hkv, N, d, page, kind, lo, hi, n_lo, causal, window):
    c = _case("", op, B, H, Hkv, N, d, page, kind, (lo, hi), n_lo, causal, window)
    del c["name"]
    return c


def _spread(lo, hi, n):
    """n lengths over [lo, hi], far apart from one another, the same for every seed."""
    return [hi] + [lo + int((hi - lo) * ((i * 0.6180339887498949) % 1.0)) for i in range(1, n)]


def _lengths(c):
    """(n_new, kv_len) of each sequence; a chunk never exceeds its cache."""
    n_new = _spread(c["n_lo"], c["N"], c["B"])
    kv = [max(a, b) for a, b in zip(_spread(c["kv_lo"], c["kv_hi"], c["B"]), n_new)]
    return n_new, kv


def _kept(c, n, kv):
    """(kept (row, key) pairs of one head, keys that any row keeps) of a chunk of n tokens at the end of kv."""
    if not c["causal"]:
        return n * kv, kv
    w = c["window"] or kv + 1
    first = kv - n  # position of the chunk's first token
    if first + 1 >= w:
        pairs = n * w
    else:
        m = min(n, w - first - 1)  # rows whose window still reaches the first key
        pairs = m * (first + 1) + m * (m - 1) // 2 + (n - m) * w
    return pairs, kv - max(0, first - w + 1)


def work(case):
    c = case
    n_new, kv = _lengths(c)
    e = 2 if c["kind"] == "bf16" else 1
    scales = 0 if c["kind"] == "bf16" else 8
    token = c["Hkv"] * (2 * c["d"] * e + scales)    # one cached token
    chunk = c["Hkv"] * 2 * c["d"] * 2               # one bf16 token of K and V
    if c["op"] == "append":
        return {"bytes": sum(n_new) * (token + chunk), "flops": 0}
    if c["op"] == "read":
        return {"bytes": sum(min(k, c["N"]) for k in kv) * token + c["B"] * c["N"] * chunk, "flops": 0}
    kept = [_kept(c, n, k) for n, k in zip(n_new, kv)]
    return {"bytes": sum(n_new) * c["H"] * c["d"] * 4 + sum(k for _, k in kept) * token,
            "flops": 4 * c["d"] * c["H"] * sum(p for p, _ in kept)}


# ---------------------------------------------------------------------------- inputs

def _codes(x):
    """(e4m3 codes, fp32 scales) of x over its last dimension."""
    amax = x.float().abs().amax(-1, keepdim=True)
    some = amax >= 2.0 ** -100
    r = torch.where(some, 448.0 / amax, torch.ones_like(amax))
    s = torch.where(some, amax / 448.0, torch.ones_like(amax))
    return (x.float() * r).to(torch.float8_e4m3fn), s.squeeze(-1)


def prepare(case, seed):
    c = case
    g = torch.Generator(device="cuda").manual_seed(seed)
    host = torch.Generator().manual_seed(seed)

    def normal(*shape):
        return torch.randn(shape, generator=g, device="cuda", dtype=torch.bfloat16)

    n_new, kv = _lengths(c)
    B, H, Hkv, N, d, page = c["B"], c["H"], c["Hkv"], c["N"], c["d"], c["page"]
    need = [-(-k // page) for k in kv]
    n_pages = sum(need) + 3
    order = torch.randperm(n_pages, generator=host, dtype=torch.int32)
    table = torch.zeros((B, max(need)), dtype=torch.int32)
    at = 0
    for b, m in enumerate(need):
        table[b, :m] = order[at:at + m]
        at += m
    shape = (n_pages, Hkv, page, d)
    # keys of one head lean the same way, as a model's do
    lean = normal(1, Hkv, 1, d)
    k, v = normal(*shape) + lean, normal(*shape)
    s = {"case": c, "table": table.cuda(), "n_new": torch.tensor(n_new, dtype=torch.int32).cuda(),
         "kv_len": torch.tensor(kv, dtype=torch.int32).cuda(), "k_scale": None, "v_scale": None}
    if c["kind"] == "e4m3":
        k, s["k_scale"] = _codes(k)
        v, s["v_scale"] = _codes(v)
        k, v = k.view(torch.uint8), v.view(torch.uint8)
    s["k"], s["v"] = k, v
    if c["op"] == "attend":
        s["q"] = normal(B, H, N, d) * 1.5
        s["o"] = torch.zeros((B, H, N, d), dtype=torch.bfloat16, device="cuda")
    elif c["op"] == "append":
        s["new_k"], s["new_v"] = normal(B, Hkv, N, d) + lean, normal(B, Hkv, N, d)
    else:
        s["out_k"] = torch.empty((B, Hkv, N, d), dtype=torch.bfloat16, device="cuda")
        s["out_v"] = torch.empty_like(s["out_k"])
    return s


# ---------------------------------------------------------------------------- the passes

def run(state):
    c = state["case"]
    if own:
        return _own(state, c)
    if c["op"] == "append":
        return _append(state, c)
    if c["op"] == "read":
        return _read(state, c)
    return _attend(state, c)


def _own(s, c):
    import block_sparse_attention_37_b200 as bsa

    if "cache" not in s:  # the handles that a program keeps beside its tensors
        s["cache"] = bsa.PagedCache(s["k"], s["v"], s["table"], s["kv_len"], s["k_scale"], s["v_scale"])
        s["dims"] = bsa.dims(c["B"], c["H"], c["N"], c["d"], 1, 1, 0)
        if c["op"] == "attend":
            s["workspace"] = torch.empty(bsa.paged_workspace_size(s["dims"], s["cache"]), dtype=torch.uint8,
                                         device="cuda")
    if c["op"] == "append":
        bsa.paged_append(s["dims"], s["cache"], s["new_k"], s["new_v"], n_new=s["n_new"])
        return _cache_of(s, c)
    if c["op"] == "read":
        bsa.paged_read(s["dims"], s["cache"], s["out_k"], s["out_v"])
        return {"k": s["out_k"], "v": s["out_v"]}
    bsa.paged_forward(s["dims"], s["cache"], s["q"], s["o"], s["workspace"], n_new=s["n_new"], causal=c["causal"],
                      window=c["window"])
    return {"o": s["o"]}


def _cache_of(s, c):
    if c["kind"] == "bf16":
        return {"k": s["k"], "v": s["v"]}
    return {"k": s["k"].view(torch.float8_e4m3fn), "v": s["v"].view(torch.float8_e4m3fn),
            "k_scale": s["k_scale"], "v_scale": s["v_scale"]}


def _append(s, c):
    n = torch.arange(c["N"], device="cuda")
    pos = (s["kv_len"] - s["n_new"])[:, None] + n                        # [B, N]
    b, i = (n < s["n_new"][:, None]).nonzero(as_tuple=True)
    at = pos[b, i]
    page, slot = s["table"][b, at // c["page"]].long(), at % c["page"]
    for name in ("k", "v"):
        x = s["new_" + name][b, :, i]                                    # [tokens, Hkv, d]
        if c["kind"] == "bf16":
            s[name][page, :, slot] = x
        else:
            codes, scale = _codes(x)
            s[name][page, :, slot] = codes.view(torch.uint8)
            s[name + "_scale"][page, :, slot] = scale
    return _cache_of(s, c)


def _gathered(s, c, name, tokens):
    """Tokens 0 .. tokens-1 of every sequence as fp32 [B, Hkv, tokens, d]; 0 past kv_len."""
    used = -(-tokens // c["page"])
    t = s["table"][:, :used].long()
    x = s[name][t].permute(0, 2, 1, 3, 4)                                # [B, Hkv, pages, page, d]
    x = x.view(torch.float8_e4m3fn).float() if c["kind"] == "e4m3" else x.float()
    if c["kind"] == "e4m3":
        x = x * s[name + "_scale"][t].permute(0, 2, 1, 3)[..., None]
    x = x.reshape(c["B"], c["Hkv"], used * c["page"], c["d"])[:, :, :tokens]
    there = torch.arange(x.shape[2], device="cuda") < s["kv_len"][:, None]
    return torch.where(there[:, None, :, None], x, torch.zeros((), device="cuda"))


def _read(s, c):
    out = {}
    for name in ("k", "v"):
        x = _gathered(s, c, name, min(c["N"], s["table"].shape[1] * c["page"]))
        s["out_" + name].zero_()
        s["out_" + name][:, :, :x.shape[2]] = x.to(torch.bfloat16)
        out[name] = s["out_" + name]
    return out


def _attend(s, c):
    B, H, Hkv, N, d = c["B"], c["H"], c["Hkv"], c["N"], c["d"]
    k, v = (_gathered(s, c, name, s["table"].shape[1] * c["page"]) for name in ("k", "v"))
    j = torch.arange(k.shape[2], device="cuda")
    n = torch.arange(N, device="cuda")
    pos = (s["kv_len"] - s["n_new"])[:, None] + n                        # [B, N]
    keep = (j < s["kv_len"][:, None])[:, None].expand(B, N, -1)
    if c["causal"]:
        keep = keep & (j <= pos[..., None])
        if c["window"]:
            keep = keep & (j > pos[..., None] - c["window"])
    keep = keep[:, None, None]                                           # [B, 1, 1, N, keys]
    q = s["q"].float().reshape(B, Hkv, H // Hkv, N, d)
    z = torch.matmul(q, k[:, :, None].transpose(-1, -2)) * d ** -0.5
    z.masked_fill_(~keep, -torch.inf)
    top = z.amax(-1, keepdim=True)
    z.sub_(torch.where(top == -torch.inf, torch.zeros_like(top), top)).exp_()
    total = z.sum(-1, keepdim=True)
    o = torch.matmul(z, v[:, :, None]) / torch.where(total > 0, total, torch.ones_like(total))
    row = (n < s["n_new"][:, None])[:, None, None, :, None]
    o = torch.where(row, o, torch.zeros((), device="cuda"))
    s["o"].copy_(o.reshape(B, H, N, d))
    return {"o": s["o"]}


# ---------------------------------------------------------------------------- from the definition, in 64 bits

def _e4m3_value(x):
    """x to the nearest value of 1 sign, 4 exponent (bias 7) and 3 mantissa bits, ties to even."""
    a = x.abs().clamp(max=448.0)
    e = torch.floor(torch.log2(a.clamp(min=2.0 ** -6)))
    step = torch.exp2(e - 3)
    return torch.copysign(torch.round(a / step) * step, x)


def exact(case, seed):
    c = case
    s = prepare(c, seed)
    n_new, kv = _lengths(c)
    page, table = c["page"], s["table"].cpu()

    def slots(b, j):
        j = torch.as_tensor(j)
        return table[b][j // page].long().cuda(), (j % page).cuda()

    def tokens(name, b, n):
        p, i = slots(b, torch.arange(n))
        x = s[name][p, :, i]
        if c["kind"] == "bf16":
            return x.double().transpose(0, 1)
        return (x.view(torch.float8_e4m3fn).double() * s[name + "_scale"][p, :, i].double()[..., None]).transpose(0, 1)

    if c["op"] == "append":
        out = {}
        for name in ("k", "v"):
            whole = s[name].double() if c["kind"] == "bf16" else s[name].view(torch.float8_e4m3fn).double()
            scale = None if c["kind"] == "bf16" else s[name + "_scale"].double()
            for b in range(c["B"]):
                x = s["new_" + name][b, :, :n_new[b]].double().transpose(0, 1)
                p, i = slots(b, torch.arange(kv[b] - n_new[b], kv[b]))
                if scale is None:
                    whole[p, :, i] = x
                else:
                    top = x.abs().amax(-1) / 448.0
                    scale[p, :, i] = top
                    whole[p, :, i] = _e4m3_value(x / top[..., None])
            out[name] = whole
            if scale is not None:
                out[name + "_scale"] = scale
        return out
    if c["op"] == "read":
        out = {}
        for name in ("k", "v"):
            out[name] = torch.zeros((c["B"], c["Hkv"], c["N"], c["d"]), dtype=torch.float64, device="cuda")
            for b in range(c["B"]):
                m = min(kv[b], c["N"])
                out[name][b, :, :m] = tokens(name, b, m)
        return out
    G = c["H"] // c["Hkv"]
    o = torch.zeros((c["B"], c["H"], c["N"], c["d"]), dtype=torch.float64, device="cuda")
    for b in range(c["B"]):
        K, V, n = tokens("k", b, kv[b]), tokens("v", b, kv[b]), n_new[b]
        pos = torch.arange(kv[b] - n, kv[b], device="cuda")[:, None]
        j = torch.arange(kv[b], device="cuda")[None]
        off = torch.zeros((n, kv[b]), dtype=torch.bool, device="cuda")
        if c["causal"]:
            off |= j > pos
            if c["window"]:
                off |= j <= pos - c["window"]
        for h in range(c["H"]):
            z = s["q"][b, h, :n].double() @ K[h // G].T / math.sqrt(c["d"])
            o[b, h, :n] = torch.softmax(z.masked_fill_(off, -torch.inf), -1) @ V[h // G]
    return {"o": o}
