"""Workloads of three operators of a paged KV cache, in plain torch and as the
library's calls:

prompt   attention of whole prompts, packed one after the other: causal,
         grouped heads, K/V as contiguous rows (not paged), optionally behind
         a prefix whose K/V rows come first.
verify   attention of several new tokens per sequence over a paged cache held
         in 4 bits (asymmetric INT4, one or two groups per head) or 8 bits
         (E4M3), with 16-bit sink tokens and an optional 16-bit window ring:
         the verify pass of speculative decoding, or a slice of a prompt.
compact  moving the kept rows of sequences into fresh blocks of every layer's
         pools, after tokens were evicted.

Each case is one call of one layer (compact: of all layers at once).
"""

import random

import torch

own = False

BS = 16  # tokens per block


# ------------------------------------------------------------------- cases
def listed():
    return [
        # three short requests of a small model: the call's own latency
        dict(name="prompt_tiny", op="prompt", lens="25,47,12", prefix="0,0,0", hq=8, hkv=2, d=64,
             dtype="fp16", fused=False),
        # a batch of requests as they arrive, odd lengths, q/k/v as views of
        # one fused projection
        dict(name="prompt_ragged", op="prompt", lens="517,1000,33,1311,250,1,764,128,2047,95,610,303",
             prefix="0,0,0,0,0,0,0,0,0,0,0,0", hq=32, hkv=8, d=128, dtype="bf16", fused=True),
        # one long document
        dict(name="prompt_8k", op="prompt", lens="8192", prefix="0", hq=32, hkv=8, d=128,
             dtype="bf16", fused=False),
        # the next turn of two conversations: 300-odd new tokens behind long
        # histories, head dim 64
        dict(name="prompt_turn", op="prompt", lens="301,277", prefix="6000,3501", hq=32, hkv=8, d=64,
             dtype="fp16", fused=False),
        # one interactive request, gamma + 1 = 6 draft tokens
        dict(name="verify_one", op="verify", batch=1, ctx_lo=4093, ctx_hi=4093, q_lo=6, q_hi=6, hq=32, hkv=8,
             d=128, dtype="bf16", mode="int4", group=128, sinks=4, window=0, len_seed=1),
        # a batch of long contexts, one group per head
        dict(name="verify_int4_16k", op="verify", batch=32, ctx_lo=16384, ctx_hi=16384, q_lo=6, q_hi=6,
             hq=32, hkv=8, d=128, dtype="bf16", mode="int4", group=128, sinks=4, window=0, len_seed=2),
        # groups of 64, 8 sinks and the last 128 tokens in 16 bits, ragged
        dict(name="verify_int4_window", op="verify", batch=24, ctx_lo=900, ctx_hi=12000, q_lo=1, q_hi=6,
             hq=32, hkv=8, d=128, dtype="fp16", mode="int4", group=64, sinks=8, window=128, len_seed=3),
        # a busy server's batch over an 8-bit cache, ragged
        dict(name="verify_fp8", op="verify", batch=64, ctx_lo=512, ctx_hi=4096, q_lo=2, q_hi=4, hq=32, hkv=8,
             d=128, dtype="bf16", mode="fp8", group=128, sinks=4, window=0, len_seed=4),
        # 512-token prompt slices that attend to the 4-bit cache before them
        dict(name="slice_int4", op="verify", batch=8, ctx_lo=4096, ctx_hi=4096, q_lo=512, q_hi=512, hq=32,
             hkv=8, d=128, dtype="bf16", mode="int4", group=128, sinks=4, window=0, len_seed=5),
        # one sequence halved, two layers
        dict(name="compact_one", op="compact", batch=1, len_lo=2051, len_hi=2051, keep=0.5, hkv=8, d=128,
             mode="bf16", layers=2, len_seed=6),
        # a batch under memory pressure keeps a third, an 8-bit cache (codes
        # and scales move together)
        dict(name="compact_fp8", op="compact", batch=16, len_lo=300, len_hi=4000, keep=0.33, hkv=8, d=128,
             mode="fp8", layers=4, len_seed=7),
        # the same over 16-bit pools of eight layers
        dict(name="compact_bf16", op="compact", batch=16, len_lo=3000, len_hi=5000, keep=0.6, hkv=8, d=128,
             mode="bf16", layers=8, len_seed=8),
    ]


def _log_int(rng, lo, hi):
    return max(lo, min(hi, int(round(lo * (hi / lo) ** rng.random()))))


def draw(rng):
    op = rng.choice(["prompt", "verify", "compact"])
    if op == "prompt":
        d = rng.choice([64, 128])
        hkv = rng.choice([1, 2, 4, 8])
        g = rng.choice([1, 2, 3, 4, 8])
        total = _log_int(rng, 24, 8000)
        n = rng.choice([1, 2, 3, 8, 20])
        lens = [max(0, int(total / n * (0.2 + 1.6 * rng.random()))) for _ in range(n)]
        if sum(lens) == 0:
            lens[0] = 1
        top = rng.choice([0, 0, 100, 1500])
        prefix = [rng.randrange(top + 1) for _ in range(n)]
        return dict(op="prompt", lens=",".join(map(str, lens)), prefix=",".join(map(str, prefix)), hq=g * hkv,
                    hkv=hkv, d=d, dtype=rng.choice(["bf16", "fp16"]), fused=rng.random() < 0.5)
    if op == "verify":
        mode = rng.choice(["int4", "int4", "fp8"])
        d = rng.choice([64, 128, 128])
        hkv = rng.choice([2, 4, 8])
        g = rng.choice([1, 2, 3, 4, 8])
        hi = _log_int(rng, 20, 12000)
        if rng.random() < 0.6:
            q_hi = rng.randint(1, 8)
            batch = _log_int(rng, 1, 48)
        else:
            q_hi = _log_int(rng, 9, 500)
            batch = _log_int(rng, 1, 6)
        lo = max(1, hi // rng.choice([1, 2, 8]))
        return dict(op="verify", batch=batch, ctx_lo=lo, ctx_hi=hi, q_lo=max(1, q_hi // 2), q_hi=q_hi, hq=g * hkv,
                    hkv=hkv, d=d, dtype=rng.choice(["bf16", "fp16"]), mode=mode,
                    group=rng.choice([64, d]) if mode == "int4" else d, sinks=rng.choice([0, 4, 8]),
                    window=rng.choice([0, 0, 64, 128]), len_seed=rng.randrange(1 << 30))
    hi = _log_int(rng, 30, 5000)
    return dict(op="compact", batch=_log_int(rng, 1, 16), len_lo=max(2, hi // 4), len_hi=hi,
                keep=round(0.1 + 0.8 * rng.random(), 3), hkv=rng.choice([1, 4, 8]), d=rng.choice([64, 128]),
                mode=rng.choice(["bf16", "fp8"]), layers=rng.randint(1, 8), len_seed=rng.randrange(1 << 30))


_TYPES = {"bf16": torch.bfloat16, "fp16": torch.float16}


def _prompt_lens(case):
    lens = [int(x) for x in case["lens"].split(",")]
    prefix = [int(x) for x in case["prefix"].split(",")]
    return lens, [p + n for p, n in zip(prefix, lens)]


def _verify_lens(case):
    r = random.Random(case["len_seed"])
    ctx = [r.randint(case["ctx_lo"], case["ctx_hi"]) for _ in range(case["batch"])]
    return [min(c, r.randint(case["q_lo"], case["q_hi"])) for c in ctx], ctx


def _compact_lens(case):
    r = random.Random(case["len_seed"])
    lens = [r.randint(case["len_lo"], case["len_hi"]) for _ in range(case["batch"])]
    return lens, [max(1, int(n * case["keep"])) for n in lens]


def work(case):
    if case["op"] == "prompt":
        lens, kv = _prompt_lens(case)
        pairs = sum(n * (t - n) + n * (n + 1) // 2 for n, t in zip(lens, kv))
        el = sum(lens) * case["hq"] * 2 + sum(kv) * case["hkv"] * 2
        return {"bytes": el * case["d"] * 2, "flops": 4 * pairs * case["hq"] * case["d"]}
    if case["op"] == "verify":
        lens, ctx = _verify_lens(case)
        pairs = sum(n * (t - n) + n * (n + 1) // 2 for n, t in zip(lens, ctx))
        d = case["d"]
        coded = d // 2 + 4 * (d // case["group"]) if case["mode"] == "int4" else d + 2
        nb = sum(lens) * case["hq"] * d * 2 * 2 + sum(-(-t // BS) for t in ctx) * 4
        for t in ctx:
            win0 = max(t - case["window"], 0) // BS * BS if case["window"] else t
            sink = min(case["sinks"], win0)
            nb += 2 * case["hkv"] * ((win0 - sink) * coded + (t - win0 + sink) * d * 2)
        return {"bytes": nb, "flops": 4 * pairs * case["hq"] * d}
    moves = sum(_compact_lens(case)[1])
    row = case["d"] * 2 if case["mode"] == "bf16" else case["d"] + 2
    return {"bytes": moves * (case["layers"] * 2 * case["hkv"] * row * 2 + 16), "flops": 0}


# ------------------------------------------------------------------ inputs
def _starts(lens, device):
    s = [0]
    for n in lens:
        s.append(s[-1] + n)
    return torch.tensor(s, dtype=torch.int32, device=device)


def _quantise(x, mode, group):
    """x [NB, H, BS, D] 16-bit -> codes, scale, zero as the cache holds them,
    a slab of blocks at a time."""
    nb, h, bs, d = x.shape
    codes = torch.empty((nb, h, bs, d // 2 if mode == "int4" else d), dtype=torch.uint8, device=x.device)
    scale = torch.empty((nb, h, bs, d // group if mode == "int4" else 1), dtype=torch.float16, device=x.device)
    zero = torch.empty_like(scale) if mode == "int4" else None
    step = max(1, (1 << 26) // (h * bs * d))
    for i in range(0, nb, step):
        f = x[i:i + step].float()
        if mode == "int4":
            f = f.view(f.shape[0], h, bs, d // group, group)
            lo, hi = f.amin(-1, keepdim=True), f.amax(-1, keepdim=True)
            s = ((hi - lo) / 15).half()
            z = (-lo / s.float()).half()
            c = torch.clamp(torch.round(f / s.float() + z.float()), 0, 15).to(torch.uint8).view(-1, h, bs, d)
            codes[i:i + step] = c[..., 0::2] | (c[..., 1::2] << 4)
            zero[i:i + step] = z[..., 0]
            scale[i:i + step] = s[..., 0]
        else:
            s = (f.abs().amax(-1, keepdim=True) / 448).half()
            c = torch.clamp(f / s.float(), -448, 448).to(torch.float8_e4m3fn)
            codes[i:i + step] = c.view(torch.uint8)
            scale[i:i + step] = s
    return codes, scale, zero


def prepare(case, seed):
    dev = torch.device("cuda")
    gen = torch.Generator(device=dev)
    gen.manual_seed(seed * 7919 + 1)

    def randn(*shape):
        return torch.randn(shape, generator=gen, device=dev, dtype=torch.float32)

    if case["op"] == "prompt":
        t = _TYPES[case["dtype"]]
        lens, kv = _prompt_lens(case)
        hq, hkv, d = case["hq"], case["hkv"], case["d"]
        T, S = sum(lens), sum(kv)
        st = {"lens": lens, "kv": kv, "q_start": _starts(lens, dev)}
        same = lens == kv
        if case["fused"] and same:
            x = randn(T, (hq + 2 * hkv) * d).to(t)
            st["q"] = x[:, :hq * d].unflatten(1, (hq, d))
            st["k"] = x[:, hq * d:(hq + hkv) * d].unflatten(1, (hkv, d))
            st["v"] = x[:, (hq + hkv) * d:].unflatten(1, (hkv, d))
        else:
            st["q"] = randn(T, hq, d).to(t)
            st["k"] = randn(S, hkv, d).to(t)
            st["v"] = randn(S, hkv, d).to(t)
        st["kv_start"] = None if same else _starts(kv, dev)
        st["scale"] = d ** -0.5
        return st

    r = random.Random(seed)
    if case["op"] == "verify":
        t = _TYPES[case["dtype"]]
        lens, ctx = _verify_lens(case)
        hq, hkv, d, B = case["hq"], case["hkv"], case["d"], case["batch"]
        need = [-(-n // BS) for n in ctx]
        mb, NB = max(need), sum(need) + 7
        order = list(range(NB))
        r.shuffle(order)
        table = torch.full((B, mb), -1, dtype=torch.int32)
        at = 0
        for b, n in enumerate(need):
            table[b, :n] = torch.tensor(order[at:at + n], dtype=torch.int32)
            at += n
        table = table.to(dev)
        lens_d = torch.tensor(ctx, dtype=torch.int32, device=dev)
        cache = {}
        ns, win = case["sinks"], case["window"]
        ring = win // BS + 1
        rows = torch.arange(B, device=dev)
        for x in ("k", "v"):
            pool = torch.empty((NB, hkv, BS, d), dtype=t, device=dev)
            for i in range(0, NB, 512):
                f = randn(min(512, NB - i), hkv, BS, d)
                hit = torch.rand(f.shape, generator=gen, device=dev) < 0.01  # 1% outliers at +-8
                pool[i:i + 512] = torch.where(hit, torch.sign(f) * 8, f).to(t)
            cache[x + "_codes"], cache[x + "_scale"], cache[x + "_zero"] = _quantise(pool, case["mode"], case["group"])
            first = table[:, 0].long().clamp(min=0)
            if ns:  # positions 0 .. ns - 1, all in block 0
                cache["sink_" + x] = pool[first][:, :, :ns].transpose(1, 2).contiguous()
            if win:  # the newest write of each ring slot
                buf = torch.zeros((B, ring, hkv, BS, d), dtype=t, device=dev)
                last = (lens_d.long() - 1) // BS
                for j in range(ring):
                    blk = last - j
                    ok = blk >= 0
                    phys = table.gather(1, blk.clamp(min=0)[:, None])[:, 0].long()
                    buf[rows[ok], (blk % ring)[ok]] = pool[phys[ok]]
                cache["win_" + x] = buf
            del pool
        st = {"cache": cache, "q": randn(sum(lens), hq, d).to(t), "q_start": _starts(lens, dev), "table": table,
              "ctx": lens_d, "scale": d ** -0.5, "max_q": max(lens), "sinks": ns, "window": win,
              "mode": case["mode"], "group": case["group"], "lens": lens}
        return st

    # compact: every sequence's kept rows go to fresh blocks
    lens, keep = _compact_lens(case)
    hkv, d = case["hkv"], case["d"]
    need = [-(-n // BS) for n in lens]
    fresh = [-(-n // BS) for n in keep]
    NB = sum(need) + sum(fresh) + 3
    order = torch.randperm(NB, generator=gen, device=dev)
    src, dst, at, to = [], [], 0, sum(need)
    for n, m, nb, fb in zip(lens, keep, need, fresh):
        kept = torch.randperm(n, generator=gen, device=dev)[:m].sort().values
        new = torch.arange(m, device=dev)
        src.append(order[at:at + nb][kept // BS] * BS + kept % BS)
        dst.append(order[to:to + fb][new // BS] * BS + new % BS)
        at, to = at + nb, to + fb
    pools = []
    for _ in range(2 * case["layers"]):
        x = torch.empty((NB, hkv, BS, d), dtype=torch.bfloat16, device=dev)
        for i in range(0, NB, 1024):
            x[i:i + 1024] = randn(min(1024, NB - i), hkv, BS, d).bfloat16()
        if case["mode"] == "bf16":
            pools.append(x)
        else:
            codes, scale, _ = _quantise(x, "fp8", d)
            pools += [codes, scale]
    return {"pools": pools, "src": torch.cat(src), "dst": torch.cat(dst)}


# -------------------------------------------------------------- plain forms
def _pad_index(start, width):
    """Row index [B, width] of each sequence's rows, and which are its own."""
    s = start.long()
    n = s[1:] - s[:-1]
    i = torch.arange(width, device=start.device)
    return s[:-1, None] + torch.minimum(i[None], (n[:, None] - 1).clamp(min=0)), i[None] < n[:, None]


def _attend(q, k, v, see, scale):
    """q [B, Lq, Hkv, G, D], k / v [B, Lk, Hkv, D] fp32, see [B, Lq, Lk]."""
    B, Lq, H, G, D = q.shape
    s = torch.matmul(q.permute(0, 2, 3, 1, 4).reshape(B, H, G * Lq, D), k.permute(0, 2, 3, 1)).mul_(scale)
    s = s.view(B, H, G, Lq, -1)
    s.masked_fill_(~see[:, None, None], float("-inf"))
    m = s.amax(-1, keepdim=True)
    s.sub_(torch.where(m == float("-inf"), torch.zeros_like(m), m)).exp_()
    l = s.sum(-1, keepdim=True)
    o = torch.matmul(s.view(B, H, G * Lq, -1), v.permute(0, 2, 1, 3)).view(B, H, G, Lq, D)
    o = torch.where(l > 0, o / l, torch.zeros_like(o))
    return o.permute(0, 3, 1, 2, 4).reshape(B, Lq, H * G, D)


def _plain_prompt(st):
    q, k, v = st["q"], st["k"], st["v"]
    hq, hkv, d = q.shape[1], k.shape[1], q.shape[2]
    Lq, Lk = max(st["lens"]), max(st["kv"])
    qi, qok = _pad_index(st["q_start"], Lq)
    kv_start = st["q_start"] if st["kv_start"] is None else st["kv_start"]
    ki, kok = _pad_index(kv_start, Lk)
    nq = (st["q_start"][1:] - st["q_start"][:-1]).long()
    nk = (kv_start[1:] - kv_start[:-1]).long()
    pos = (nk - nq)[:, None] + torch.arange(Lq, device=q.device)
    see = (torch.arange(Lk, device=q.device)[None, None] <= pos[:, :, None]) & kok[:, None]
    o = _attend(q[qi.clamp(max=q.shape[0] - 1)].float().view(-1, Lq, hkv, hq // hkv, d),
                k[ki.clamp(max=k.shape[0] - 1)].float(), v[ki.clamp(max=v.shape[0] - 1)].float(), see, st["scale"])
    return o[qok].to(q.dtype)


def _dequant(codes, scale, zero, mode, group):
    """[..., D] values of codes [..., D/2 or D] fp32."""
    if mode == "fp8":
        return codes.view(torch.float8_e4m3fn).float() * scale.float()
    c = torch.stack((codes & 15, codes >> 4), -1).flatten(-2).float().unflatten(-1, (-1, group))
    return ((c - zero.float()[..., None]) * scale.float()[..., None]).flatten(-2)


def _plain_verify(st):
    q, cache, table = st["q"], st["cache"], st["table"]
    B, mb = table.shape
    hq, d = q.shape[1], q.shape[2]
    hkv = cache["k_codes"].shape[1]
    ctx = st["ctx"].long()
    S = mb * BS
    t = torch.arange(S, device=q.device)
    phys = table.long().clamp(min=0)
    win0 = (ctx - st["window"]).clamp(min=0) // BS * BS if st["window"] else ctx

    def rows(x):
        zero = cache[x + "_zero"]
        f = _dequant(cache[x + "_codes"][phys], cache[x + "_scale"][phys], None if zero is None else zero[phys],
                     st["mode"], st["group"])
        f = f.transpose(2, 3).reshape(B, S, hkv, d)
        if st["sinks"]:
            n = min(st["sinks"], S)
            f[:, :n] = cache["sink_" + x][:, :n].float()
        if st["window"]:
            ring = cache["win_" + x].transpose(2, 3)  # [B, ring, BS, H, D]
            n = min(ring.shape[1], mb)
            blk = (win0 // BS)[:, None] + torch.arange(n, device=q.device)  # the window's blocks
            blk = torch.minimum(blk, ((ctx - 1) // BS)[:, None])
            b = torch.arange(B, device=q.device)[:, None]
            f.view(B, mb, BS, hkv, d)[b, blk] = ring[b, blk % ring.shape[1]].float()
        return f

    Lq = st["max_q"]
    qi, qok = _pad_index(st["q_start"], Lq)
    nq = (st["q_start"][1:] - st["q_start"][:-1]).long()
    pos = (ctx - nq)[:, None] + torch.arange(Lq, device=q.device)
    see = (t[None, None] <= pos[:, :, None]) & (t[None, None] < ctx[:, None, None])
    o = _attend(q[qi.clamp(max=q.shape[0] - 1)].float().view(B, Lq, hkv, hq // hkv, d), rows("k"), rows("v"), see,
                st["scale"])
    return o[qok].to(q.dtype)


def _plain_compact(st):
    src, dst = st["src"], st["dst"]
    for p in st["pools"]:
        p[dst // BS, :, dst % BS] = p[src // BS, :, src % BS]
    return _values(st["pools"])


def _values(pools):
    """The pools as run() returns them: 8-bit codes as the values they stand for."""
    return [p.view(torch.float8_e4m3fn) if p.dtype == torch.uint8 else p for p in pools]


# ------------------------------------------------------------------ the pass
def run(st):
    if own:
        import paged_kv_cache_13_gb300 as pkv

        if "pools" in st:
            pkv.pkv_move_rows(st["pools"], st["src"], st["dst"])
            return _values(st["pools"])
        q = st["q"]
        if "out" not in st:  # the output and the workspace that a program keeps
            st["out"] = torch.empty(q.shape, dtype=q.dtype, device=q.device)
            if "cache" in st:
                kc = st["cache"]["k_codes"]
                n = pkv.pkv_multi_query_quant_workspace_bytes(st["ctx"].shape[0], q.shape[1], kc.shape[1], q.shape[2],
                                                              st["table"].shape[1], st["max_q"])
            else:
                n = pkv.pkv_prompt_attention_workspace_bytes(st["q_start"].shape[0] - 1, q.shape[0], st["k"].shape[0],
                                                             q.shape[1], st["k"].shape[1], q.shape[2])
            st["ws"] = torch.empty(n, dtype=torch.uint8, device=q.device) if n else None
        if "cache" in st:
            pkv.pkv_paged_attention_multi_query_quant(
                q, st["q_start"], st["cache"], st["sinks"], st["table"], st["ctx"], st["scale"], st["out"],
                st["max_q"], st["mode"], group_size=st["group"], workspace=st["ws"], window=st["window"])
        else:
            pkv.pkv_prompt_attention(q, st["k"], st["v"], st["q_start"], st["scale"], st["out"],
                                     kv_start=st["kv_start"], workspace=st["ws"])
        return st["out"]
    if "pools" in st:
        return _plain_compact(st)
    return _plain_verify(st) if "cache" in st else _plain_prompt(st)


# ---------------------------------------------------------------- 64 bits
def _exact_rows(q, k, v, scale):
    """One sequence: q [Lq, Hq, D], k / v [Lk, Hkv, D] float64, the queries
    being the last Lq of the Lk positions."""
    Lq, hq, _ = q.shape
    Lk, hkv, _ = k.shape
    out = torch.empty_like(q)
    hide = torch.ones((Lq, Lk), dtype=torch.bool, device=q.device).triu(Lk - Lq + 1)
    for h in range(hq):
        kh = h // (hq // hkv)
        s = q[:, h] @ k[:, kh].T * scale
        s[hide] = -float("inf")
        out[:, h] = torch.softmax(s, -1) @ v[:, kh]
    return out


def exact(case, seed):
    st = prepare(case, seed)
    if case["op"] == "compact":
        outs = []
        for p in _values(st["pools"]):
            e = p.double()
            e[st["dst"] // BS, :, st["dst"] % BS] = p[st["src"] // BS, :, st["src"] % BS].double()
            outs.append(e)
        return outs
    q = st["q"].double()
    outs = []
    if case["op"] == "prompt":
        lens, kv = _prompt_lens(case)
        a = b = 0
        for n, m in zip(lens, kv):
            if n:
                outs.append(_exact_rows(q[a:a + n], st["k"][b:b + m].double(), st["v"][b:b + m].double(), st["scale"]))
            a, b = a + n, b + m
        return torch.cat(outs)
    lens, ctx = _verify_lens(case)
    cache, a = st["cache"], 0
    for b, (n, c) in enumerate(zip(lens, ctx)):
        blocks = st["table"][b, :-(-c // BS)].long()
        kv = []
        for x in ("k", "v"):
            codes = cache[x + "_codes"][blocks].permute(0, 2, 1, 3).flatten(0, 1)[:c]  # [c, H, .]
            s = cache[x + "_scale"][blocks].permute(0, 2, 1, 3).flatten(0, 1)[:c].double()
            if case["mode"] == "int4":
                z = cache[x + "_zero"][blocks].permute(0, 2, 1, 3).flatten(0, 1)[:c].double()
                val = torch.empty(codes.shape[:2] + (2 * codes.shape[2],), dtype=torch.float64, device=q.device)
                val[..., 0::2] = (codes % 16).double()
                val[..., 1::2] = (codes // 16).double()
                g = case["group"]
                val = (val - z.repeat_interleave(g, -1)) * s.repeat_interleave(g, -1)
            else:
                val = codes.view(torch.float8_e4m3fn).double() * s
            m = min(c, case["sinks"])
            if m:
                val[:m] = cache["sink_" + x][b, :m].double()
            if case["window"]:
                w0 = max(c - case["window"], 0) // BS * BS
                p = torch.arange(w0, c, device=q.device)
                ring = cache["win_" + x].shape[1]
                val[p] = cache["win_" + x][b, p // BS % ring, :, p % BS].double()
            kv.append(val)
        outs.append(_exact_rows(q[a:a + n], kv[0], kv[1], st["scale"]))
        a += n
    return torch.cat(outs)
