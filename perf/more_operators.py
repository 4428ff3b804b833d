"""A prompt through a layer in 8-bit integers: the operators as they are measured.

  quant  quant_int8           rows of activations to int8 with one fp32 scale each, optionally of
                              silu(gate) * up, optionally per expert with live-row counts
  mm     scaled_mm_int8       int8 x int8 product with a scale for each token and each channel
  rope   qk_norm_rope_axes    RMS norm of query and key heads and the rotation by positions on
                              several axes (time, height, width)
  attn   attention_packed     attention of packed prompts of different lengths over their own
                              16-bit keys and values, grouped heads

`run` computes the plain form in elementary torch operations, or calls the library (`own`).
"""
import math
import random

import torch

own = False

DTYPES = {"bf16": torch.bfloat16, "fp16": torch.float16}
FLOOR = 1e-10          # the library's floor of a row's largest magnitude


# ------------------------------------------------------------------------------------ the cases

def listed():
    return [
        # the input of a 8320-token prompt's QKV product
        dict(name="quant_prefill", op="quant", E=0, M=8320, K=5376, silu=False, mean=0, dtype="bf16"),
        # a decode batch routed to 32 experts of 128-row slabs: their down projections' input
        dict(name="quant_experts", op="quant", E=32, M=128, K=2048, silu=True, mean=32, dtype="fp16"),
        # one decode step of 16 sequences, gate or up projection: the weights' stream
        dict(name="mm_decode", op="mm", E=0, M=16, N=14336, K=4096, mean=0, bias=False, dtype="bf16"),
        # a short prompt's down projection, odd rows, with bias
        dict(name="mm_short_prompt", op="mm", E=0, M=333, N=5376, K=14336, mean=0, bias=True, dtype="fp16"),
        # the experts' down projections of that decode batch
        dict(name="mm_experts", op="mm", E=32, M=128, N=7168, K=2048, mean=32, bias=False, dtype="bf16"),
        # the QKV product of the 8320-token prompt
        dict(name="mm_prefill", op="mm", E=0, M=8320, N=21504, K=5376, mean=0, bias=False, dtype="bf16"),
        # a decode step of 16 sequences far into their texts: three equal positions a token
        dict(name="rope_decode", op="rope", T=16, Hq=32, Hk=8, Hx=8, D=128, rot=128, axes=3, mixed=False,
             norm=True, pairs=False, far=131072, dtype="bf16"),
        # the query and key heads of a video of 8320 patches; the axes alternate pair by pair
        dict(name="rope_video", op="rope", T=8320, Hq=56, Hk=56, Hx=56, D=128, rot=128, axes=3, mixed=True,
             norm=True, pairs=False, far=1024, dtype="bf16"),
        # a single short question: latency
        dict(name="attn_short", op="attn", B=1, lo=77, hi=77, mix=1, Hq=32, Hkv=8, D=128, causal=True,
             window=0, dtype="bf16"),
        # the 8320-token prompt
        dict(name="attn_prompt", op="attn", B=1, lo=8320, hi=8320, mix=2, Hq=56, Hkv=56, D=128, causal=True,
             window=0, dtype="bf16"),
        # prompts of many lengths packed one behind the other, eight key heads
        dict(name="attn_texts", op="attn", B=13, lo=0, hi=3001, mix=3, Hq=32, Hkv=8, D=128, causal=True,
             window=0, dtype="bf16"),
        # patches of pictures of different sizes, each seeing its whole picture
        dict(name="attn_pictures", op="attn", B=7, lo=256, hi=2500, mix=4, Hq=16, Hkv=16, D=64, causal=False,
             window=0, dtype="fp16"),
    ]


def draw(rng):
    def log(lo, hi):
        return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))

    op = rng.choice(["quant", "mm", "mm", "rope", "attn", "attn"])
    dtype = rng.choice(["bf16", "bf16", "fp16"])
    if op == "quant":
        silu = rng.random() < 0.5
        E = rng.choice([0, 0, log(1, 32)])
        K = 8 * log(1, 336 if silu else 672)
        M = log(1, 256 if E else 8320)
        return dict(op=op, E=E, M=M, K=K, silu=silu, mean=log(1, M) if E else 0, dtype=dtype)
    if op == "mm":
        E = rng.choice([0, 0, 0, log(1, 32)])
        M = log(1, 128 if E else 8320)
        N = 8 * log(1, 896 if E else 2688)
        K = 16 * log(1, 128 if E else 896)
        if M * N * K > 8320 * 21504 * 5376:
            M = max(1, 8320 * 21504 * 5376 // (N * K))
        return dict(op=op, E=E, M=M, N=N, K=K, mean=log(1, M) if E else 0, bias=rng.random() < 0.4, dtype=dtype)
    D = rng.choice([64, 128, 128])
    if op == "rope":
        Hk = rng.choice([1, 2, 4, 7, 8, 16])
        return dict(op=op, T=log(1, 8320), Hq=Hk * rng.choice([1, 2, 4, 7]), Hk=Hk, Hx=rng.choice([0, Hk]), D=D,
                    rot=rng.choice([D, D, D // 2, 16]), axes=rng.choice([2, 3, 3, 4]), mixed=rng.random() < 0.5,
                    norm=rng.random() < 0.7, pairs=rng.random() < 0.4, far=rng.choice([64, 1024, 131072]),
                    dtype=dtype)
    Hkv = rng.choice([1, 2, 4, 7, 8])
    causal = rng.random() < 0.7
    hi = log(1, 8320)
    B = rng.randint(1, max(1, min(16, 16640 // hi)))
    return dict(op=op, B=B, lo=rng.choice([0, 1, hi]) if B > 1 else hi, hi=hi, mix=rng.randrange(1 << 30),
                Hq=Hkv * rng.choice([1, 2, 4, 5]), Hkv=Hkv, D=D, causal=causal,
                window=log(1, 4096) if causal and rng.random() < 0.4 else 0, dtype=dtype)


def _lengths(case):
    """The prompts' lengths, from the case alone; with lo = 0 one of them has no tokens, one a single one."""
    r = random.Random(case["mix"])
    n = [r.randint(case["lo"], case["hi"]) for _ in range(case["B"])]
    if case["lo"] == 0 and case["B"] > 2:
        n[0], n[1] = 0, 1
    if sum(n) == 0:
        n[-1] = 1
    return n


def _rows(case):
    """The experts' live rows, from the case alone; few tokens leave experts idle, the last one never is."""
    r = random.Random(case["E"] * 1000003 + case["M"])
    live = [min(case["M"], max(0, int(round(r.gauss(case["mean"], math.sqrt(case["mean"])))))) for _ in range(case["E"])]
    live[-1:] = [max(1, live[-1])] if live else []
    return live


def _pairs(case):
    """(query, key) pairs that a head sees."""
    w = case["window"]
    total = 0
    for n in _lengths(case):
        if not case["causal"]:
            total += n * n
        elif w and n > w:
            total += w * (w + 1) // 2 + (n - w) * w
        else:
            total += n * (n + 1) // 2
    return total


def work(case):
    op = case["op"]
    if op == "quant":
        rows = sum(_rows(case)) if case["E"] else case["M"]
        read = (4 if case["silu"] else 2) * case["K"]
        return {"bytes": rows * (read + case["K"] + 4), "flops": rows * case["K"] * (9 if case["silu"] else 3)}
    if op == "mm":
        live = _rows(case) if case["E"] else [case["M"]]
        N, K = case["N"], case["K"]
        return {"bytes": sum(m * (K + 2 * N + 4) + (N * (K + 4) if m else 0) for m in live)
                + (2 * N if case["bias"] else 0), "flops": 2 * sum(live) * N * K}
    if op == "rope":
        T, row = case["T"], (case["Hq"] + case["Hk"]) * case["D"]
        flops = T * row * ((4 if case["norm"] else 0) + 3 * case["rot"] / case["D"])
        return {"bytes": T * (4 * row + 4 * case["axes"] + 4 * case["rot"]) + (4 * case["D"] if case["norm"] else 0),
                "flops": flops}
    T = sum(_lengths(case))
    return {"bytes": T * (case["Hq"] * (4 * case["D"] + 4) + case["Hkv"] * 4 * case["D"]),
            "flops": 4 * _pairs(case) * case["Hq"] * case["D"]}


# ------------------------------------------------------------------------------------ the inputs

def prepare(case, seed):
    dev = torch.device("cuda")
    gen = torch.Generator(device=dev).manual_seed(seed)
    dt = DTYPES[case["dtype"]]
    op = case["op"]
    s = {"case": case, "dt": dt}

    def normal(*shape):
        return torch.randn(*shape, generator=gen, device=dev)

    def uniform(*shape):
        return torch.rand(*shape, generator=gen, device=dev)

    if op in ("quant", "mm"):
        E, M, K = case["E"], case["M"], case["K"]
        lead = (E,) if E else ()
        s["rows"] = torch.tensor(_rows(case), dtype=torch.int32, device=dev) if E else None
        if E:
            s["live"] = torch.arange(M, device=dev) < s["rows"][:, None]
        if op == "quant":
            x = normal(*lead, M, 2 * K if case["silu"] else K)
            x *= 1.0 + 15.0 * (uniform(x.shape[-1]) < 0.01)       # a few outlier channels
            s["x"] = x.to(dt)
            s["q"] = torch.zeros(*lead, M, K, dtype=torch.int8, device=dev)
            s["scales"] = torch.zeros(*lead, M, dtype=torch.float32, device=dev)
            return s
        N = case["N"]

        def codes(*shape):      # rows of a normal distribution whose largest value lies about four deviations out
            c = torch.empty(*shape, dtype=torch.int8, device=dev)
            flat = c.view(-1)
            for i in range(0, flat.numel(), 1 << 26):      # in pieces: bounded memory
                m = min(1 << 26, flat.numel() - i)
                flat[i:i + m] = (normal(m) * 32).round().clamp(-127, 127).to(torch.int8)
            return c

        s["a"], s["b"] = codes(*lead, M, K), codes(*lead, N, K)
        s["sa"] = (0.5 + uniform(*lead, M)) * (4 / 127)
        s["sb"] = (0.5 + uniform(*lead, N)) * (0.08 / 127)
        s["bias"] = normal(N).to(dt) if case["bias"] else None
        s["c"] = torch.zeros(*lead, M, N, dtype=dt, device=dev)
        return s
    D = case["D"]
    if op == "rope":
        T, heads, half, axes = case["T"], case["Hq"] + case["Hk"], case["rot"] // 2, case["axes"]
        x = normal(T, (heads + case["Hx"]) * D)
        x *= 1.0 + 7.0 * (uniform((heads + case["Hx"]) * D) < 0.02)
        s["x"] = x.to(dt)
        s["y"] = torch.empty(T, heads * D, dtype=dt, device=dev)
        s["positions"] = torch.randint(0, case["far"], (axes, T), generator=gen, device=dev, dtype=torch.int32)
        # the pair's axis: in turn, or one section behind the other with a shorter first one
        first = max(1, half // (axes + 1))
        s["axes"] = [i % axes for i in range(half)] if case["mixed"] else \
            [0 if i < first else 1 + (i - first) * (axes - 1) // (half - first) for i in range(half)]
        freq = 10000.0 ** (-torch.arange(half, device=dev, dtype=torch.float64) / half)
        angle = torch.arange(case["far"], device=dev, dtype=torch.float64)[:, None] * freq
        s["cos_sin"] = torch.cat([angle.cos(), angle.sin()], 1).float()
        s["wq"] = (1 + 0.2 * normal(D)).to(dt) if case["norm"] else None
        s["wk"] = (1 + 0.2 * normal(D)).to(dt) if case["norm"] else None
        return s
    n = _lengths(case)
    T, Hq, H = sum(n), case["Hq"], case["Hkv"]
    s["n"] = n
    s["cu"] = torch.tensor([0] + n, device=dev).cumsum(0).int()
    rows = normal(T, (Hq + 2 * H) * D)
    rows[:, :Hq * D] *= (0.5 + 3.0 * uniform(Hq, 1) ** 3).expand(Hq, D).reshape(-1)     # some heads look at a few tokens only
    rows = rows.to(dt)
    q, k, v = rows.split([Hq * D, H * D, H * D], 1)       # columns of one projection
    s["q"], s["k"], s["v"] = q.unflatten(1, (Hq, D)), k.unflatten(1, (H, D)), v.unflatten(1, (H, D))
    return s


# ------------------------------------------------------------------------------------ one pass

def run(s):
    return (_run_own if own else _run_plain)(s)


def _run_own(s):
    from column_scaled_gemm_amd import fp8sm
    c = s["case"]
    if c["op"] == "quant":
        return fp8sm.quant_int8(s["x"], fuse_silu_mul=c["silu"], rows=s["rows"], q=s["q"], scales=s["scales"])
    if c["op"] == "mm":
        return fp8sm.scaled_mm_int8(s["a"], s["b"], s["sa"], s["sb"], rows=s["rows"], c=s["c"], bias=s["bias"])
    if c["op"] == "rope":
        return fp8sm.qk_norm_rope_axes(s["x"], c["Hq"], c["Hk"], c["D"], s["positions"], s["cos_sin"], s["axes"],
                                       q_weight=s["wq"], k_weight=s["wk"], eps=1e-6, interleaved=c["pairs"],
                                       out=s["y"])
    return fp8sm.attention_packed(s["q"], s["k"], s["v"], s["cu"], causal=c["causal"], window=c["window"],
                                  return_lse=True)


def _run_plain(s):
    return {"quant": _plain_quant, "mm": _plain_mm, "rope": _plain_rope, "attn": _plain_attn}[s["case"]["op"]](s)


def _plain_quant(s):
    x = s["x"].float()
    if s["case"]["silu"]:
        gate, up = x.chunk(2, -1)
        # a code changes at a border: the exponential rounded once to 32 bits
        x = gate / (1.0 + torch.exp(-gate.double()).float()) * up
    top = x.abs().amax(-1).clamp(min=FLOOR)
    unit = torch.full_like(top, 127.0)          # (a tensor: division by, or of, a number takes its reciprocal)
    q = (x * (unit / top)[..., None]).round().clamp(-127, 127).to(torch.int8)
    scale = top / unit
    if s["rows"] is None:
        s["q"].copy_(q)
        s["scales"].copy_(scale)
    else:
        s["q"].copy_(torch.where(s["live"][..., None], q, s["q"]))
        s["scales"].copy_(torch.where(s["live"], scale, s["scales"]))
    return s["q"], s["scales"]


def _plain_mm(s):
    y = torch.matmul(s["a"].float(), s["b"].float().transpose(-1, -2).contiguous())
    y = y * s["sa"][..., None] * s["sb"][..., None, :]
    if s["bias"] is not None:
        y = y + s["bias"].float()
    y = y.to(s["dt"])
    s["c"].copy_(y if s["rows"] is None else torch.where(s["live"][..., None], y, s["c"]))
    return s["c"]


def _plain_rope(s):
    c = s["case"]
    T, Hq, Hk, D, rot = c["T"], c["Hq"], c["Hk"], c["D"], c["rot"]
    half = rot // 2
    x = s["x"][:, :(Hq + Hk) * D].float().view(T, Hq + Hk, D)
    if s["wq"] is not None:
        w = torch.cat([s["wq"].float().expand(Hq, D), s["wk"].float().expand(Hk, D)])
        x = x * torch.rsqrt((x * x).mean(-1, keepdim=True) + 1e-6) * w
    column = torch.arange(half, device=x.device)
    row = s["positions"].long()[torch.tensor(s["axes"], device=x.device)].t()       # [T, half]
    cos, sin = s["cos_sin"][row, column][:, None], s["cos_sin"][row, column + half][:, None]
    if c["pairs"]:
        a, b = x[..., 0:rot:2], x[..., 1:rot:2]
        turned = torch.stack([a * cos - b * sin, b * cos + a * sin], -1).flatten(-2)
    else:
        a, b = x[..., :half], x[..., half:rot]
        turned = torch.cat([a * cos - b * sin, b * cos + a * sin], -1)
    s["y"].copy_(torch.cat([turned, x[..., rot:]], -1).view(T, -1))
    return s["y"]


def _plain_attn(s):
    """The prompts as a padded batch."""
    c = s["case"]
    Hq, H, D, w = c["Hq"], c["Hkv"], c["D"], c["window"]
    B, L, G = c["B"], max(s["n"]), c["Hq"] // c["Hkv"]
    cu = s["cu"].long()
    n = cu[1:] - cu[:-1]
    at = torch.arange(L, device=cu.device)
    held = at < n[:, None]                                         # [B, L]
    row = torch.where(held, cu[:-1, None] + at, 0)

    def padded(x):                                                 # [T, heads, D] -> [B, heads, L, D]
        return x[row].float().transpose(1, 2)

    k = padded(s["k"]).transpose(2, 3).contiguous()
    v = padded(s["v"]).contiguous()
    q = padded(s["q"]).reshape(B, H, G * L, D) * D ** -0.5
    hide = ~held[:, None, :]
    if c["causal"]:
        hide = hide | (at > at[:, None])
        if w:
            hide = hide | (at <= at[:, None] - w)
    a = torch.matmul(q, k).view(B, H, G, L, L)
    a.masked_fill_(hide[:, None, None], float("-inf"))
    top = a.amax(-1, keepdim=True)
    top = torch.where(top == float("-inf"), 0.0, top)              # padded rows see nothing
    a = a.sub_(top).exp_()
    total = a.sum(-1, keepdim=True)
    o = torch.matmul(a.view(B, H, G * L, L), v).view(B, H, G, L, D) / total
    lse = (top + total.log())[..., 0]
    o = o.view(B, Hq, L, D).transpose(1, 2)[held]
    return o.to(s["dt"]), lse.view(B, Hq, L).transpose(1, 2)[held]


# ------------------------------------------------------------------------------------ in 64 bits

def exact(case, seed):
    s = prepare(case, seed)
    op = case["op"]
    if op == "quant":
        x = s["x"].double()
        if case["silu"]:
            K = case["K"]
            x = x[..., :K] * torch.sigmoid(x[..., :K]) * x[..., K:]
        scale = x.abs().max(-1).values.clamp(min=FLOOR) / 127
        # the codes are whole numbers of 32-bit roundings: nothing in 64 bits to set beside them
        return None, scale if s["rows"] is None else scale * s["live"]
    if op == "mm":
        a, b = s["a"], s["b"]
        if not case["E"]:
            a, b = a[None], b[None]
        out = []
        for e in range(a.shape[0]):
            y = a[e].double() @ b[e].double().T
            y *= s["sa"].view(a.shape[0], -1)[e].double()[:, None]
            y *= s["sb"].view(a.shape[0], -1)[e].double()
            if s["bias"] is not None:
                y += s["bias"].double()
            if case["E"]:
                y[s["rows"][e]:] = 0
            out.append(y)
        return torch.stack(out) if case["E"] else out[0]
    if op == "rope":
        Hq, Hk, D, half = case["Hq"], case["Hk"], case["D"], case["rot"] // 2
        x = s["x"].double()[:, :(Hq + Hk) * D].unflatten(1, (Hq + Hk, D))
        if case["norm"]:
            x = x / (x.square().sum(2, keepdim=True) / D + 1e-6).sqrt()
            x[:, :Hq] *= s["wq"].double()
            x[:, Hq:] *= s["wk"].double()
        z = x.clone()
        for i, axis in enumerate(s["axes"]):
            p = s["positions"][axis].long()
            cos, sin = (s["cos_sin"][p, j].double()[:, None] for j in (i, i + half))
            m, k = (2 * i, 2 * i + 1) if case["pairs"] else (i, i + half)
            z[..., m] = x[..., m] * cos - x[..., k] * sin
            z[..., k] = x[..., k] * cos + x[..., m] * sin
        return z.flatten(1)
    Hq, H, w = case["Hq"], case["Hkv"], case["window"]
    out = torch.empty(s["q"].shape, dtype=torch.float64, device="cuda")
    lse = torch.empty(s["q"].shape[:2], dtype=torch.float64, device="cuda")
    at = 0
    for n in s["n"]:
        rows = slice(at, at + n)
        t = torch.arange(n, device="cuda")
        far = t[:, None] - t
        hidden = (far < 0) | (far >= w) if w else far < 0
        for h in range(Hq if n else 0):
            g = h // (Hq // H)
            a = s["q"][rows, h].double() @ s["k"][rows, g].double().T.contiguous() / math.sqrt(case["D"])
            if case["causal"]:
                a[hidden] = float("-inf")
            lse[rows, h] = torch.logsumexp(a, 1)
            out[rows, h] = torch.exp(a - lse[rows, h, None]) @ s["v"][rows, g].double()
        at += n
    return out, lse
