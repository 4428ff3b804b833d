"""The operators between the QKV projection and the output projection, as they are measured.

  rope   qk_norm_rope     RMS norm of every query and key head and the position rotation, one pass
  write  kv_cache_write   keys and values quantised into a paged E4M3 cache (one power-of-two scale
                          for each block of tokens and head); the touched blocks are read back
  read   kv_cache_read    cached tokens gathered and widened to 16 bits
  attn   attention_cache  causal attention of ragged queries over that cache

A cache is four tensors: K codes [blocks, Hkv, block, D], V codes [blocks, Hkv, block/16, D, 16]
and their biased exponents [blocks, Hkv] (a value is code * 2^(byte - 127)).  Sequence b of a batch
has its tokens' rows cu[b] .. cu[b+1]-1 in the ragged activations, `lens[b]` cached tokens once they
are written (they are the last ones), and the block numbers table[b].

`run` computes the plain form in elementary torch operations, or calls the library (`own`).
"""
import math
import random

import torch

own = False

DTYPES = {"bf16": torch.bfloat16, "fp16": torch.float16}


# ------------------------------------------------------------------------------------ the cases

def listed():
    return [
        # one decode step of 16 sequences far into their texts: latency
        dict(name="rope_decode", op="rope", T=16, Hq=32, Hk=8, Hx=8, D=128, rot=128, norm=True,
             interleaved=False, dtype="bf16", far=131072),
        # the rows of the 8320-token QKV product (56 query, key and value heads of 128)
        dict(name="rope_prefill", op="rope", T=8320, Hq=56, Hk=56, Hx=56, D=128, rot=128, norm=True,
             interleaved=False, dtype="bf16", far=16384),
        # odd token count, half of each small head rotated in adjacent pairs, no norm
        dict(name="rope_partial", op="rope", T=1001, Hq=7, Hk=7, Hx=7, D=64, rot=32, norm=False,
             interleaved=True, dtype="fp16", far=4096),
        # one token appended to each of 64 sequences: blocks that hold old tokens
        dict(name="write_append", op="write", B=64, n_lo=1, n_hi=1, len_lo=100, len_hi=4000, mix=1,
             Hkv=8, D=128, block=16, dtype="bf16"),
        # the keys and values of that 8320-token prompt
        dict(name="write_prefill", op="write", B=1, n_lo=8320, n_hi=8320, len_lo=8320, len_hi=8320,
             mix=2, Hkv=56, D=128, block=64, dtype="bf16"),
        # a few ragged prefixes taken out of the cache again
        dict(name="read_ragged", op="read", B=5, n_lo=33, n_hi=4000, len_lo=4000, len_hi=5000, mix=3,
             Hkv=7, D=64, block=32, dtype="fp16"),
        # a batch's whole caches, e.g. to hand them on to another worker
        dict(name="read_batch", op="read", B=16, n_lo=4096, n_hi=4096, len_lo=4096, len_hi=4096,
             mix=4, Hkv=8, D=128, block=64, dtype="bf16"),
        # one user's next token: latency
        dict(name="attn_decode_one", op="attn", B=1, n_lo=1, n_hi=1, len_lo=1000, len_hi=1000, mix=5,
             Hq=32, Hkv=8, D=128, block=16, window=0, dtype="bf16"),
        # a full decode batch of ragged lengths: the cache's stream
        dict(name="attn_decode_batch", op="attn", B=64, n_lo=1, n_hi=1, len_lo=500, len_hi=16384,
             mix=6, Hq=32, Hkv=8, D=128, block=64, window=0, dtype="bf16"),
        # two very long texts, four drafted tokens each
        dict(name="attn_decode_long", op="attn", B=2, n_lo=4, n_hi=4, len_lo=131000, len_hi=131072,
             mix=7, Hq=64, Hkv=8, D=128, block=64, window=0, dtype="bf16"),
        # a mixed step: prompt pieces, single tokens and sequences without any, sliding window
        dict(name="attn_mixed_window", op="attn", B=9, n_lo=0, n_hi=1500, len_lo=1500, len_hi=6001,
             mix=8, Hq=14, Hkv=2, D=64, block=32, window=1000, dtype="fp16"),
        # the 8320-token prompt itself
        dict(name="attn_prefill", op="attn", B=1, n_lo=8320, n_hi=8320, len_lo=8320, len_hi=8320,
             mix=9, Hq=56, Hkv=56, D=128, block=64, window=0, dtype="bf16"),
    ]


def draw(rng):
    def log(lo, hi):
        return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))

    op = rng.choice(["rope", "write", "read", "attn", "attn", "attn"])
    dtype = rng.choice(["bf16", "bf16", "fp16"])
    D = rng.choice([64, 128, 128])
    if op == "rope":
        Hk = rng.choice([1, 2, 4, 7, 8, 16])
        Hq = Hk * rng.choice([1, 2, 4, 7])
        rot = rng.choice([D, D, D // 2, 16])
        return dict(op=op, T=log(1, 8320), Hq=Hq, Hk=Hk, Hx=rng.choice([0, Hk]), D=D, rot=rot,
                    norm=rng.random() < 0.7, interleaved=rng.random() < 0.4, dtype=dtype,
                    far=rng.choice([1024, 16384, 262144]))
    block = rng.choice([16, 32, 64, 128])
    Hkv = rng.choice([1, 2, 4, 7, 8])
    mix = rng.randrange(1 << 30)
    if op == "attn":
        kind = rng.choice(["decode", "decode", "draft", "piece", "mixed"])
        B = log(1, 64) if kind in ("decode", "draft") else log(1, 9)
        n_lo, n_hi = {"decode": (1, 1), "draft": (1, rng.randint(2, 9)),
                      "piece": (lambda n: (max(1, n // 2), n))(log(17, 2000)),
                      "mixed": (0, log(2, 1500))}[kind]
        len_hi = max(n_hi, log(1, 16384 if kind in ("decode", "draft") else 8192))
        return dict(op=op, B=B, n_lo=n_lo, n_hi=n_hi, len_lo=max(1, n_hi, len_hi // rng.choice([1, 4, 30])),
                    len_hi=max(1, n_hi, len_hi), mix=mix, Hq=Hkv * rng.choice([1, 2, 4, 5, 8]), Hkv=Hkv,
                    D=D, block=block, window=rng.choice([0, 0, log(1, 4096)]), dtype=dtype)
    B = log(1, 64)
    n_hi = max(1, log(1, 16384) // B)
    n_lo = rng.choice([0, 1, n_hi])
    len_hi = n_hi + log(1, 4000) - 1
    return dict(op=op, B=B, n_lo=min(n_lo, n_hi), n_hi=n_hi, len_lo=max(1, n_hi, len_hi // 3), len_hi=max(1, len_hi),
                mix=mix, Hkv=Hkv, D=D, block=block, dtype=dtype)


def _lengths(case):
    """Each sequence's new tokens and cached tokens, from the case alone."""
    r = random.Random(case["mix"])
    B = case["B"]
    n = [r.randint(case["n_lo"], case["n_hi"]) for _ in range(B)]
    length = [r.randint(case["len_lo"], case["len_hi"]) for _ in range(B)]
    if case["n_lo"] == 0 and B > 2:      # a sequence without new tokens and one with a single one
        n[0], n[1] = 0, 1
    if sum(n) == 0:
        n[-1] = 1
    return n, [max(a, b) for a, b in zip(n, length)]


def _tail(n, length, block):
    """Tokens of each sequence from the start of the first block that its new tokens touch."""
    return [L - (L - k) // block * block if k else 0 for k, L in zip(n, length)]


def _pairs(case):
    """Visible (query, key) pairs of one head."""
    n, length = _lengths(case)
    w = case["window"]
    total = 0
    for k, L in zip(n, length):
        for p in (range(L - k, L) if k <= 64 else ()):
            total += min(p + 1, w) if w else p + 1
        if k > 64:
            full = k * (L - k) + k * (k + 1) // 2
            if w:
                # of the positions at and behind the window, what lies before it
                lo = max(L - k, w)
                m = max(0, L - lo)
                full -= sum((lo + 1 - w, L - w)) * m // 2 if m else 0
            total += full
    return total


def work(case):
    op = case["op"]
    if op == "rope":
        row = (case["Hq"] + case["Hk"]) * case["D"]
        flops = case["T"] * row * ((4 if case["norm"] else 0) + 3 * case["rot"] / case["D"])
        return {"bytes": case["T"] * (4 * row + 4 + 4 * case["rot"]) + (4 * case["D"] if case["norm"] else 0),
                "flops": flops}
    n, length = _lengths(case)
    row = case["Hkv"] * case["D"]
    if op == "write":
        # new values in; the touched blocks' codes out, in again and widened
        tail = sum(_tail(n, length, case["block"]))
        return {"bytes": sum(n) * row * 4 + tail * row * (2 + 4), "flops": sum(n) * row * 6 + tail * row * 2}
    if op == "read":
        return {"bytes": sum(n) * row * (2 + 4), "flops": sum(n) * row * 2}
    w = case["window"]
    seen = sum(min(L, w + k - 1) if w else L for k, L in zip(n, length) if k)
    return {"bytes": sum(n) * case["Hq"] * (4 * case["D"] + 4) + seen * row * 2,
            "flops": 4 * _pairs(case) * case["Hq"] * case["D"]}


# ------------------------------------------------------------------------------------ the inputs

def _inputs(case, seed):
    dev = torch.device("cuda")
    gen = torch.Generator(device=dev).manual_seed(seed)
    dt = DTYPES[case["dtype"]]

    def normal(*shape):
        return torch.randn(*shape, generator=gen, device=dev)

    s = {"case": case, "dt": dt}
    D = case["D"]
    if case["op"] == "rope":
        T, heads = case["T"], case["Hq"] + case["Hk"]
        # rows of a QKV product: a few outlier channels, the value heads behind
        gain = 1.0 + 7.0 * (torch.rand((heads + case["Hx"]) * D, generator=gen, device=dev) < 0.02)
        x = normal(T, (heads + case["Hx"]) * D)
        x *= gain
        s["x"] = x.to(dt)
        s["y"] = torch.empty(T, heads * D, dtype=dt, device=dev)
        s["pos"] = torch.randint(0, case["far"], (T,), generator=gen, device=dev, dtype=torch.int32)
        half = case["rot"] // 2
        freq = 10000.0 ** (-torch.arange(half, device=dev, dtype=torch.float64) / half)
        ang = torch.arange(case["far"], device=dev, dtype=torch.float64)[:, None] * freq
        s["cos_sin"] = torch.cat([ang.cos(), ang.sin()], 1).float()
        s["wq"] = (1 + 0.2 * normal(D)).to(dt) if case["norm"] else None
        s["wk"] = (1 + 0.2 * normal(D)).to(dt) if case["norm"] else None
        return s
    n, length = _lengths(case)
    B, H, block = case["B"], case["Hkv"], case["block"]
    s["n"], s["len"] = n, length
    need = [-(-L // block) for L in length]
    spare = 3
    blocks = sum(need) + spare
    order = torch.randperm(blocks, generator=gen, device=dev).int()
    table = torch.zeros(B, max(need), dtype=torch.int32, device=dev)
    at = 0
    for b in range(B):
        table[b, :need[b]] = order[at:at + need[b]]
        at += need[b]
    s["table"] = table
    s["cu"] = torch.tensor([0] + n, device=dev).cumsum(0).int()
    s["lens"] = torch.tensor(length, dtype=torch.int32, device=dev)
    s["total"] = sum(n)

    def codes(*shape):
        c = torch.empty(*shape, dtype=torch.uint8, device=dev)
        flat = c.view(-1)
        for i in range(0, flat.numel(), 1 << 26):      # in pieces: the draws are 32-bit
            m = min(1 << 26, flat.numel() - i)
            flat[i:i + m] = (normal(m) * 80).clamp(-448, 448).to(torch.float8_e4m3fn).view(torch.uint8)
        return c

    def exponents():
        # blocks of unit scale within a binade or two: 448 * 2^-7 = 3.5, 2^-6: 7
        return torch.randint(119, 122, (blocks, H), generator=gen, device=dev, dtype=torch.int32).to(torch.uint8)

    s["cache"] = (codes(blocks, H, block, D), codes(blocks, H, block // 16, D, 16), exponents(), exponents())
    if case["op"] == "write":
        rows = normal(s["total"], 2 * H * D)
        rows[:, ::97] *= 6.0                              # outlier channels
        rows = rows.to(dt)
        s["k"] = rows[:, :H * D].unflatten(1, (H, D))     # slices of the projection's rows
        s["v"] = rows[:, H * D:].unflatten(1, (H, D))
        tail = _tail(n, length, block)
        s["tail"] = tail
        s["cu_tail"] = torch.tensor([0] + tail, device=dev).cumsum(0).int()
        s["tail_total"] = sum(tail)
    elif case["op"] == "attn":
        q = normal(s["total"], case["Hq"], D)
        # some heads look at a few tokens only
        q *= 0.5 + 3.0 * torch.rand(case["Hq"], 1, generator=gen, device=dev) ** 3
        s["q"] = q.to(dt)
        s["max_q"], s["max_kv"] = max(n), max(length)
    return s


def prepare(case, seed):
    s = _inputs(case, seed)
    if own and case["op"] != "rope":
        from column_scaled_gemm_amd import fp8sm
        s["cache"] = fp8sm.KVCache(*s["cache"])
    return s


# ------------------------------------------------------------------------------------ one pass

def run(s):
    return (_run_own if own else _run_plain)(s)


def _run_own(s):
    from column_scaled_gemm_amd import fp8sm
    c = s["case"]
    if c["op"] == "rope":
        return fp8sm.qk_norm_rope(s["x"], c["Hq"], c["Hk"], c["D"], s["pos"], s["cos_sin"],
                                  q_weight=s["wq"], k_weight=s["wk"], eps=1e-6,
                                  interleaved=c["interleaved"], out=s["y"])
    if c["op"] == "write":
        fp8sm.kv_cache_write(s["k"], s["v"], s["cache"], s["cu"], s["lens"], s["table"])
        return fp8sm.kv_cache_read(s["cache"], s["cu_tail"], s["lens"], s["table"], s["tail_total"],
                                   dtype=s["dt"])
    if c["op"] == "read":
        return fp8sm.kv_cache_read(s["cache"], s["cu"], s["lens"], s["table"], s["total"], dtype=s["dt"])
    return fp8sm.attention_cache(s["q"], s["cache"], s["cu"], s["lens"], s["table"], s["max_q"],
                                 max_kv=s["max_kv"], causal=True, window=c["window"], return_lse=True)


def _run_plain(s):
    c = s["case"]
    return {"rope": _plain_rope, "write": _plain_write, "read": _plain_read, "attn": _plain_attn}[c["op"]](s)


def _plain_rope(s):
    c = s["case"]
    T, Hq, Hk, D, rot = c["T"], c["Hq"], c["Hk"], c["D"], c["rot"]
    half = rot // 2
    x = s["x"][:, :(Hq + Hk) * D].float().view(T, Hq + Hk, D)
    if s["wq"] is not None:
        w = torch.cat([s["wq"].float().expand(Hq, D), s["wk"].float().expand(Hk, D)])
        x = x * torch.rsqrt((x * x).mean(-1, keepdim=True) + 1e-6) * w
    table = s["cos_sin"][s["pos"].long()]
    cos, sin = table[:, None, :half], table[:, None, half:]
    if c["interleaved"]:
        a, b = x[..., 0:rot:2], x[..., 1:rot:2]
        turned = torch.stack([a * cos - b * sin, b * cos + a * sin], -1).flatten(-2)
    else:
        a, b = x[..., :half], x[..., half:rot]
        turned = torch.cat([a * cos - b * sin, b * cos + a * sin], -1)
    s["y"].copy_(torch.cat([turned, x[..., rot:]], -1).view(T, -1))
    return s["y"]


def _decode(codes):
    return codes.view(torch.float8_e4m3fn).float()


def _scale(exponent):
    return torch.exp2(exponent.float() - 127)


def _encode(x, exponent):
    """Codes of x for a block exponent (int tensor that broadcasts)."""
    y = (x * torch.exp2(127 - exponent.float())).clamp(-448, 448)
    return y.to(torch.float8_e4m3fn).view(torch.uint8)


def _exponent(amax):
    """Biased exponent of the smallest power of two that holds amax / 448."""
    t = amax.clamp(min=1e-10) / 448
    m, e = torch.frexp(t)                       # t = m 2^e, m in [0.5, 1)
    return torch.where(m == 0.5, e - 1, e) + 127


def _block_keys(cache, which, pages):
    """[pages, H, block, D] codes, whichever way the cache holds them."""
    x = cache[which][pages]
    if which == 1:
        x = x.permute(0, 1, 2, 4, 3).flatten(2, 3)
    return x


def _plain_write(s):
    c = s["case"]
    block, H, D = c["block"], c["Hkv"], c["D"]
    at = 0
    for b in range(c["B"]):
        n, length = s["n"][b], s["len"][b]
        if n == 0:
            continue
        first, last = (length - n) // block, (length - 1) // block
        pages = s["table"][b, first:last + 1].long()
        old = length - n - first * block        # tokens that the first block holds already
        slots = (last - first + 1) * block
        fresh = torch.zeros(slots, dtype=torch.bool, device=pages.device)
        fresh[old:old + n] = True
        held = torch.zeros_like(fresh)
        held[:old] = True
        fresh = fresh.view(-1, 1, block, 1)
        held = held.view(-1, 1, block, 1)
        for which, x in ((0, s["k"]), (1, s["v"])):
            new = torch.zeros(slots, H, D, device=pages.device)
            new[old:old + n] = x[at:at + n].float()
            new = new.view(-1, block, H, D).transpose(1, 2)
            codes = _block_keys(s["cache"], which, pages)
            before = s["cache"][2 + which][pages].int()
            e = _exponent(new.abs().amax((2, 3)))
            e = torch.where(held.view(-1, 1, block).any(2), torch.maximum(e, before), e)
            again = _encode(_decode(codes) * torch.exp2((before - e).float())[:, :, None, None], torch.full_like(e, 127)[:, :, None, None])
            codes = torch.where(fresh, _encode(new, e[:, :, None, None]), torch.where(held, again, codes))
            if which == 1:
                codes = codes.unflatten(2, (block // 16, 16)).permute(0, 1, 2, 4, 3)
            s["cache"][which][pages] = codes
            s["cache"][2 + which][pages] = e.to(torch.uint8)
        at += n
    return _gather(s, s["tail"], s["tail_total"])


def _gather(s, n, total):
    """The last n[b] tokens of every sequence, widened."""
    c = s["case"]
    block = c["block"]
    out = []
    for which in (0, 1):
        parts = []
        for b in range(c["B"]):
            if n[b] == 0:
                continue
            length = s["len"][b]
            first = (length - n[b]) // block
            pages = s["table"][b, first:(length - 1) // block + 1].long()
            x = _decode(_block_keys(s["cache"], which, pages)) * _scale(s["cache"][2 + which][pages])[:, :, None, None]
            x = x.transpose(1, 2).flatten(0, 1)
            start = length - n[b] - first * block
            parts.append(x[start:start + n[b]].to(s["dt"]))
        out.append(torch.cat(parts))
    return tuple(out)


def _plain_read(s):
    return _gather(s, s["n"], s["total"])


def _plain_attn(s):
    c = s["case"]
    Hq, H, D, block, w = c["Hq"], c["Hkv"], c["D"], c["block"], c["window"]
    G = Hq // H
    scale = D ** -0.5
    out = torch.empty_like(s["q"])
    lse = torch.empty(s["total"], Hq, device=out.device)
    at = 0
    for b in range(c["B"]):
        n, length = s["n"][b], s["len"][b]
        if n == 0:
            continue
        lo = max(0, length - n - w + 1) // block * block if w else 0     # no query sees before it
        pages = s["table"][b, lo // block:(length - 1) // block + 1].long()
        kv = []
        for which in (0, 1):
            x = _decode(_block_keys(s["cache"], which, pages)) * _scale(s["cache"][2 + which][pages])[:, :, None, None]
            kv.append(x.transpose(0, 1).flatten(1, 2)[:, :length - lo])
        k, v = kv
        col = torch.arange(lo, length, device=out.device)
        step = max(1, min(n, (1 << 30) // (length - lo) // G))            # rows at a time: bounded memory
        for i in range(0, n, step):
            j = min(n, i + step)
            pos = torch.arange(length - n + i, length - n + j, device=out.device)[:, None]
            hide = col > pos
            if w:
                hide |= col <= pos - w
            for h in range(H) if (j - i) * G * (length - lo) * H > 1 << 28 else (slice(None),):
                kh, vh = (k[h][None], v[h][None]) if isinstance(h, int) else (k, v)
                q = s["q"][at + i:at + j].float().view(j - i, H, G, D).permute(1, 2, 0, 3)
                q = q[h][None] if isinstance(h, int) else q
                m = kh.shape[0]
                a = torch.matmul(q.reshape(m, G * (j - i), D) * scale, kh.transpose(1, 2).contiguous())
                a = a.view(m, G, j - i, -1).masked_fill_(hide, float("-inf"))
                top = a.amax(-1, keepdim=True)
                a = a.sub_(top).exp_()
                total = a.sum(-1, keepdim=True)
                o = torch.matmul(a.view(m, G * (j - i), -1), vh.contiguous()).view(m, G, j - i, D) / total
                heads = slice(h * G, h * G + G) if isinstance(h, int) else slice(None)
                out[at + i:at + j, heads] = o.permute(2, 0, 1, 3).reshape(j - i, m * G, D).to(out.dtype)
                lse[at + i:at + j, heads] = (top + total.log())[..., 0].permute(2, 0, 1).reshape(j - i, m * G)
        at += n
    return out, lse


# ------------------------------------------------------------------------------------ in 64 bits

def _value_of_code():
    """The 256 E4M3 values from their bit fields."""
    vals = []
    for code in range(256):
        e, m = code >> 3 & 15, code & 7
        v = m * 2.0 ** -9 if e == 0 else (8 + m) * 2.0 ** (e - 10)
        v = float("nan") if e == 15 and m == 7 else v
        vals.append(-v if code & 128 else v)
    return torch.tensor(vals, dtype=torch.float64, device="cuda")


def _round_e4m3(y):
    """y rounded to the nearest E4M3 value (ties to the even one), |y| <= 448."""
    step = torch.exp2(torch.floor(torch.log2(y.abs().clamp(min=2.0 ** -6))) - 3)
    return torch.round(y / step) * step


def _tokens(s, b, which, lo, hi, head=slice(None)):
    """Values of tokens lo .. hi-1 of sequence b, in 64 bits: [tokens, H, D]."""
    c = s["case"]
    t = torch.arange(lo, hi, device="cuda")
    page = s["table"][b].long()[t // c["block"]]
    slot = t % c["block"]
    cache = s["cache"]
    x = cache[0][page, :, slot] if which == 0 else cache[1][page, :, slot // 16, :, slot % 16]
    return s["value"][x[:, head].long()] * torch.exp2(cache[2 + which][page][:, head].double() - 127)[..., None]


def exact(case, seed):
    s = _inputs(case, seed)
    op = case["op"]
    if op == "rope":
        Hq, Hk, D, rot = case["Hq"], case["Hk"], case["D"], case["rot"]
        half = rot // 2
        x = s["x"].double()[:, :(Hq + Hk) * D].unflatten(1, (Hq + Hk, D))
        if case["norm"]:
            x = x / (x.square().sum(2, keepdim=True) / D + 1e-6).sqrt()
            x[:, :Hq] *= s["wq"].double()
            x[:, Hq:] *= s["wk"].double()
        z = x.clone()
        first = torch.arange(half, device="cuda") * (2 if case["interleaved"] else 1)
        second = first + (1 if case["interleaved"] else half)
        turn = s["cos_sin"].double()[s["pos"].long()]
        cos, sin = turn[:, None, :half], turn[:, None, half:]
        z[..., first] = x[..., first] * cos - x[..., second] * sin
        z[..., second] = x[..., second] * cos + x[..., first] * sin
        return z.flatten(1)
    s["value"] = _value_of_code()
    n, length = s["n"], s["len"]
    if op == "read":
        return tuple(torch.cat([_tokens(s, b, which, length[b] - n[b], length[b]) for b in range(case["B"])])
                     for which in (0, 1))
    if op == "write":
        return tuple(_exact_write(s, which) for which in (0, 1))
    out, lse = [], []
    Hq, H, w = case["Hq"], case["Hkv"], case["window"]
    at = 0
    for b in range(case["B"]):
        k, L = n[b], length[b]
        if k == 0:
            continue
        o = torch.empty(k, Hq, case["D"], dtype=torch.float64, device="cuda")
        z = torch.empty(k, Hq, dtype=torch.float64, device="cuda")
        for g in range(H):
            keys, vals = (_tokens(s, b, which, 0, L, slice(g, g + 1))[:, 0] for which in (0, 1))
            for h in range(g * (Hq // H), (g + 1) * (Hq // H)):
                a = s["q"][at:at + k, h].double() @ keys.T.contiguous() / math.sqrt(case["D"])
                far = torch.arange(L - k, L, device="cuda")[:, None] - torch.arange(L, device="cuda")
                a[(far < 0) | (far >= w) if w else far < 0] = float("-inf")
                z[:, h] = torch.logsumexp(a, 1)
                o[:, h] = torch.exp(a - z[:, h, None]) @ vals
        out.append(o)
        lse.append(z)
        at += k
    return torch.cat(out), torch.cat(lse)


def _exact_write(s, which):
    c = s["case"]
    block = c["block"]
    x = (s["k"], s["v"])[which].double()
    out = []
    at = 0
    for b in range(c["B"]):
        n, L = s["n"][b], s["len"][b]
        for p in range((L - n) // block * block, L if n else 0, block):
            lo, hi = max(p, L - n), min(p + block, L)
            new = x[at + lo - (L - n):at + hi - (L - n)]
            # the smallest e with 448 * 2^e >= every new value
            need = new.abs().amax((0, 2)).clamp(min=1e-10) / 448
            e = torch.ceil(torch.log2(need))
            e = torch.where(448 * torch.exp2(e - 1) >= need * 448, e - 1, e)
            if lo > p:                                    # old tokens keep a block's exponent from falling
                page = s["table"][b, p // block].long()
                e = torch.maximum(e, s["cache"][2 + which][page].double() - 127)
                old = _tokens(s, b, which, p, lo)
                unit = torch.exp2(e)[None, :, None]
                out.append(_round_e4m3((old / unit).clamp(-448, 448)) * unit)
            unit = torch.exp2(e)[None, :, None]
            out.append(_round_e4m3((new / unit).clamp(-448, 448)) * unit)
        at += n
    return torch.cat(out)
