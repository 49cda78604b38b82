"""The four-bit token operators as they are measured: cases, inputs, plain forms and exact values.

Three operators of a transformer block whose weights, keys and values are
held in four bits: `linear` (matrix product of few rows with such weights),
`store` (tokens quantised into the pages of a cache, and read back) and
`attend` (attention over such a cache). With `own` false, run() computes them
in elementary torch operations in 32 bits; with `own` true it makes the
package's calls.

The format: 32 neighbours share one scale byte s, each is a code of a sign,
two exponent bits and one of mantissa (0, 0.5, 1, 1.5, 2, 3, 4, 6), and a
value is code * 2^(s - 127). A byte holds two codes, the earlier one low.
"""
import math

import torch

own = False

DEVICE = "cuda"
TYPES = {"bf16": torch.bfloat16, "f32": torch.float32}


def listed():
    return [
        # one token's output projection with its residual: latency of a serving step
        dict(name="linear_one_token", op="linear", M=1, K=1024, N=1024, act="none", residual=True, out="bf16"),
        # one token through the first feed-forward layer of a large block
        dict(name="linear_one_token_wide", op="linear", M=1, K=4096, N=16384, act="gelu", residual=False, out="bf16"),
        # a decoding step of 13 sequences through a second feed-forward layer, a ragged number of features out
        dict(name="linear_decode_step", op="linear", M=13, K=16384, N=4095, act="none", residual=False, out="f32"),
        # the prompted rows of a few crops through the first feed-forward layer
        dict(name="linear_prompt_rows", op="linear", M=37, K=1024, N=4096, act="gelu", residual=False, out="bf16"),
        # every prompt row of an image and a half, float32 residual stream
        dict(name="linear_many_rows", op="linear", M=128, K=8192, N=8192, act="none", residual=True, out="f32"),
        # the newest token of 48 sequences, grouped heads
        dict(name="store_new_tokens", op="store", B=48, T=1, Hk=8, D=128, page=64, start=1024, ragged=True,
             dtype="bf16"),
        # 64 crops of 24 x 24 tokens behind 5 leading tokens, each crop a sequence of its own
        dict(name="store_image_tokens", op="store", B=64, T=581, Hk=16, D=64, page=32, start=0, ragged=False,
             dtype="bf16"),
        # one prompt row against one image's tokens: latency
        dict(name="attend_one_row", op="attend", B=1, Tq=1, Hq=16, Hk=16, D=64, S=576, page=64, causal=False,
             ragged=False),
        # 37 prompt sets of up to 80 rows, each against the 48 x 48 tokens of its own stored image
        dict(name="attend_prompt_sets", op="attend", B=37, Tq=80, Hq=16, Hk=16, D=64, S=2304, page=64, causal=False,
             ragged=True),
        # a decoding step of 48 sequences, some slots of the batch idle
        dict(name="attend_decode", op="attend", B=48, Tq=1, Hq=32, Hk=8, D=128, S=8192, page=64, causal=True,
             ragged=True),
        # a decoding step of one very long sequence
        dict(name="attend_long", op="attend", B=1, Tq=1, Hq=32, Hk=8, D=128, S=262144, page=128, causal=True,
             ragged=False),
        # a piece of a prompt of each of four sequences, behind long caches
        dict(name="attend_piece", op="attend", B=4, Tq=128, Hq=32, Hk=8, D=128, S=16384, page=64, causal=True,
             ragged=True),
    ]


def _spread(rng, low, high):
    """A whole number of low .. high, spread over its logarithm."""
    return max(low, min(high, int(round(math.exp(rng.uniform(math.log(low), math.log(high)))))))


def draw(rng):
    op = rng.choice(("linear", "store", "attend"))
    if op == "linear":
        # rows from one token to a batch of prompt rows; whole groups of 32 along K
        M = _spread(rng, 1, 128)
        K = 32 * _spread(rng, 8, 512)
        N = _spread(rng, 16, min(16384, 8192 * 8192 // K))
        return dict(op=op, M=M, K=K, N=N, act=rng.choice(("none", "relu", "gelu", "quick_gelu", "silu")),
                    residual=rng.random() < 0.5, out=rng.choice(("bf16", "bf16", "f32")))
    D = rng.choice((64, 128))
    Hk = _spread(rng, 1, 16)
    B = _spread(rng, 1, 64)
    page = rng.choice((32, 64, 64, 128, 256))
    if op == "store":
        dtype = rng.choice(("bf16", "bf16", "f32"))
        most = 64 * 581 * 16 * 64 // (Hk * D * B * (2 if dtype == "f32" else 1))
        return dict(op=op, B=B, T=_spread(rng, 1, max(1, min(4096, most))), Hk=Hk, D=D, page=page,
                    start=rng.choice((0, _spread(rng, 1, 4096))), ragged=rng.random() < 0.7, dtype=dtype)
    Hq = Hk * rng.choice((1, 2, 4, 7, 8))
    S = _spread(rng, 1, 65536)
    Tq = 1 if rng.random() < 0.4 else min(S, _spread(rng, 2, 256))
    # no more key values and no more products than the largest listed cases have
    while B * S * Hk * D > 48 * 8192 * 8 * 128 or B * Tq * Hq * S * D > 4 * 128 * 32 * 16384 * 128:
        B, S, Tq = max(1, B * 3 // 4), max(1, S * 3 // 4), max(1, Tq * 3 // 4)
    return dict(op=op, B=B, Tq=Tq, Hq=Hq, Hk=Hk, D=D, S=S, page=page, causal=rng.random() < 0.6,
                ragged=rng.random() < 0.7)


def _lengths(case):
    """Tokens of each sequence in the cache: from half the space to all of it;
    the fifth slot of a ragged batch is idle and holds none."""
    if not case["ragged"]:
        return [case["S"]] * case["B"]
    low = max(case["Tq"], case["S"] // 2)
    return [0 if b == 4 else low + (7919 * (b + 1)) % max(1, case["S"] - low + 1) for b in range(case["B"])]


def _query_lengths(case):
    """Rows in use of each sequence: all in decoding and causal passes, a padded batch otherwise."""
    if case["causal"] or not case["ragged"]:
        return [case["Tq"]] * case["B"]
    return [1 + (104729 * (b + 1)) % case["Tq"] for b in range(case["B"])]


def _starts(case):
    """Tokens that a sequence's cache holds before the new ones."""
    if not case["ragged"]:
        return [case["start"]] * case["B"]
    return [case["start"] // 2 + (7919 * (b + 1)) % (case["start"] // 2 + 1) for b in range(case["B"])]


def _counts(case):
    """New tokens of each sequence."""
    if not case["ragged"]:
        return [case["T"]] * case["B"]
    return [1 + (104729 * (b + 1)) % case["T"] for b in range(case["B"])]


def _quantised(v):
    """Codes [..., n/2] and scale bytes [..., n/32] of values [..., n] in float32."""
    g = v.unflatten(-1, (-1, 32))
    a = g.abs().amax(-1, keepdim=True)
    # 2^e with a < 7 2^e: the exponent of a, one more where its mantissa reaches 1.75, less two
    e = (((a.view(torch.int32) + 0x200000) >> 23) - 127 - 2).clamp(-125, 125)
    unit = ((e + 127) << 23).view(torch.float32)
    r = g.abs() / unit
    c = ((r > 0.25).to(torch.uint8) + (r >= 0.75) + (r > 1.25) + (r >= 1.75) + (r > 2.5) + (r >= 3.5) + (r > 5))
    c = (c | ((g < 0).to(torch.uint8) << 3)).flatten(-2)
    return c[..., 0::2] | (c[..., 1::2] << 4), (e + 127).to(torch.uint8).flatten(-2)


def _values(codes, scales):
    """Values [..., n] in float32 of codes [..., n/2] and scale bytes [..., n/32]."""
    table = torch.tensor([0, 0.5, 1, 1.5, 2, 3, 4, 6, -0.0, -0.5, -1, -1.5, -2, -3, -4, -6], device=codes.device)
    both = torch.stack((codes & 15, codes >> 4), -1).flatten(-2)
    unit = (scales.to(torch.int32) << 23).view(torch.float32)
    return (table[both.int()].unflatten(-1, (-1, 32)) * unit[..., None]).flatten(-2)


def _cache(case, g, tokens, filled):
    """An empty cache, or one of normally distributed keys and values, with a
    page table in no order: room for `tokens` tokens of each sequence."""
    B, Hk, D, page = (case[k] for k in ("B", "Hk", "D", "page"))
    L = (tokens + page - 1) // page
    n = B * L + 3  # some pages belong to none of these sequences
    codes = torch.zeros(n, 2, Hk, page, D // 2, dtype=torch.uint8, device=DEVICE)
    scales = torch.full((n, 2, Hk, page, D // 32), 127, dtype=torch.uint8, device=DEVICE)
    if filled:
        step = max(1, (1 << 26) // (2 * Hk * page * D))
        for p in range(0, n, step):
            v = torch.randn(min(step, n - p), 2, Hk, page, D, generator=g, device=DEVICE)
            codes[p:p + step], scales[p:p + step] = _quantised(v)
    table = torch.randperm(n, generator=g, device=DEVICE)[:B * L].reshape(B, L).to(torch.int32)
    return codes, scales, table


def prepare(case, seed):
    g = torch.Generator(device=DEVICE)
    g.manual_seed(seed)

    def randn(*shape, scale=1.0, dtype=torch.bfloat16):
        return (torch.randn(*shape, generator=g, device=DEVICE) * scale).to(dtype)

    def ints(values):
        return torch.tensor(values, dtype=torch.int32, device=DEVICE)

    s = dict(case)
    if case["op"] == "linear":
        M, K, N = case["M"], case["K"], case["N"]
        s["x"] = randn(M, K)
        s["codes"], s["scales"] = _quantised(randn(N, K, scale=K ** -0.5, dtype=torch.float32))
        s["b"] = randn(N, scale=0.1)
        s["r"] = randn(M, N, dtype=TYPES[case["out"]]) if case["residual"] else None
    elif case["op"] == "store":
        B, T, Hk, D = (case[k] for k in ("B", "T", "Hk", "D"))
        rows = randn(B, T, 2, Hk, D, dtype=TYPES[case["dtype"]])  # one projection's rows: keys, then values
        s["k"], s["v"] = rows[:, :, 0], rows[:, :, 1]
        s["codes"], s["scales"], s["table"] = _cache(case, g, case["start"] + T, False)
        s["at"], s["count"] = ints(_starts(case)), ints(_counts(case))
        s["ko"], s["vo"] = (torch.zeros(B, T, Hk, D, dtype=torch.bfloat16, device=DEVICE) for _ in range(2))
    else:
        B, Tq, Hq, D = (case[k] for k in ("B", "Tq", "Hq", "D"))
        s["q"] = randn(B, Tq, Hq, D)
        s["codes"], s["scales"], s["table"] = _cache(case, g, case["S"], True)
        s["length"], s["q_len"] = ints(_lengths(case)), ints(_query_lengths(case))
        s["out"] = torch.zeros(B, Tq, Hq, D, dtype=torch.bfloat16, device=DEVICE)
    return s


def _act(y, kind):
    if kind == "relu":
        return torch.where(y > 0, y, 0.0)
    if kind == "gelu":
        return 0.5 * y * (1 + torch.erf(y * 0.5 ** 0.5))
    if kind == "quick_gelu":
        return y / (1 + torch.exp(-1.702 * y))
    if kind == "silu":
        return y / (1 + torch.exp(-y))
    return y


def _linear(s):
    w = _values(s["codes"], s["scales"])
    y = _act(torch.matmul(s["x"].float(), w.t()) + s["b"].float(), s["act"])
    if s["r"] is not None:
        y = y + s["r"].float()
    return y.to(TYPES[s["out"]])


def _places(s):
    """Pages and rows [B, T] of the new tokens, and which of them there are."""
    t = torch.arange(s["T"], device=s["table"].device)
    at = s["at"].long()[:, None] + t
    page = torch.gather(s["table"].long(), 1, (at // s["page"]).clamp_max(s["table"].shape[1] - 1))
    return page, at % s["page"], t < s["count"][:, None]


def _store(s):
    page, row, there = _places(s)
    pages, rows = page[there], row[there]
    out = []
    for i, x in enumerate((s["k"], s["v"])):
        codes, scales = _quantised(x[there].float())
        s["codes"][pages, i, :, rows], s["scales"][pages, i, :, rows] = codes, scales
    for i in range(2):
        y = _values(s["codes"][page, i, :, row], s["scales"][page, i, :, row])
        out.append(torch.where(there[..., None, None], y, 0.0).to(torch.bfloat16))
    return tuple(out)


def _attend(s):
    B, Tq, Hq, Hk, D, S = (s[k] for k in ("B", "Tq", "Hq", "Hk", "D", "S"))
    G = Hq // Hk
    n, t_n = s["length"].long(), s["q_len"].long()
    pages = s["table"].long()
    y = torch.zeros(B, Hk, Tq * G, D, device=s["q"].device)
    q = s["q"].float().reshape(B, Tq, Hk, G, D).permute(0, 2, 1, 3, 4).reshape(B, Hk, Tq * G, D) * D ** -0.5
    j = torch.arange(S, device=n.device)
    seen = (j < n[:, None])[:, None]                                                 # [B, 1, S]
    if s["causal"]:
        t = torch.arange(Tq, device=n.device).repeat_interleave(G)
        seen = seen & (j <= (n - t_n)[:, None, None] + t[:, None])
    k, v = (_values(s["codes"][pages, i], s["scales"][pages, i]).transpose(1, 2).flatten(2, 3)[:, :, :S]
            for i in range(2))                                                       # [B, Hk, S, D]
    score = torch.where(seen[:, None], torch.matmul(q, k.transpose(2, 3)), -math.inf)
    top = score.amax(-1, keepdim=True)
    p = torch.exp(score - torch.where(top > -math.inf, top, 0.0))
    y = torch.matmul(p, v) / p.sum(-1, keepdim=True).clamp_min(1e-30)
    y = y.reshape(B, Hk, Tq, G, D).permute(0, 2, 1, 3, 4).reshape(B, Tq, Hq, D)
    used = torch.arange(Tq, device=y.device) < t_n[:, None]
    return torch.where(used[..., None, None], y, 0.0).to(torch.bfloat16)


def run(state):
    s = state
    if own:
        import prompt_conditioned_keypoint_amd as gkd
        if s["op"] == "linear":
            return gkd.linear_fp4(s["x"], s["codes"], s["scales"], bias=s["b"], residual=s["r"], act=s["act"],
                                  out_dtype=TYPES[s["out"]])
        if s["op"] == "store":
            gkd.cache_append(s["k"], s["v"], s["codes"], s["scales"], s["table"], start=s["at"], count=s["count"])
            return gkd.cache_read(s["codes"], s["scales"], s["table"], s["T"], start=s["at"], count=s["count"],
                                  k_out=s["ko"], v_out=s["vo"])
        return gkd.cache_attention(s["q"], s["codes"], s["scales"], s["table"], length=s["length"],
                                   q_len=s["q_len"], causal=s["causal"], out=s["out"])
    return {"linear": _linear, "store": _store, "attend": _attend}[s["op"]](s)


def work(case):
    c = case
    if c["op"] == "linear":
        e = 4 if c["out"] == "f32" else 2
        moved = (2 * (c["M"] * c["K"] + c["N"]) + c["N"] * c["K"] * 17 // 32 +
                 e * c["M"] * c["N"] * (2 if c["residual"] else 1))
        return {"bytes": moved, "flops": 2 * c["M"] * c["N"] * c["K"]}
    if c["op"] == "store":
        n = sum(_counts(c)) * 2 * c["Hk"] * c["D"]
        # values in, codes and scales out and in again, bfloat16 out
        return {"bytes": n * (4 if c["dtype"] == "f32" else 2) + 2 * (n * 17 // 32) + 2 * n, "flops": 4 * n}
    rows, keys, pairs = 0, 0, 0
    for n, t in zip(_lengths(c), _query_lengths(c)):
        rows += t
        keys += n
        pairs += t * (n - t) + t * (t + 1) // 2 if c["causal"] and n >= t else t * n
    moved = 4 * rows * c["Hq"] * c["D"] + 2 * keys * c["Hk"] * c["D"] * 17 // 32
    return {"bytes": moved, "flops": 4 * pairs * c["Hq"] * c["D"]}


def _exact_values(codes, scales):
    """Values in float64 from the bits: (-1)^sign (mantissa / 2) 2^(exponent of the code and scale)."""
    nibbles = torch.cat(((codes & 15)[..., None], (codes >> 4)[..., None]), -1).reshape(*codes.shape[:-1], -1).long()
    exponent, half = (nibbles >> 1) & 3, (nibbles & 1).double() / 2
    size = torch.where(exponent == 0, half, (1 + half) * 2.0 ** (exponent - 1).double())
    size = torch.where(nibbles >= 8, -size, size)
    unit = torch.pow(2.0, scales.double() - 127)
    return size * unit.repeat_interleave(32, -1)


def _exact_rounded(v):
    """What is left of values in float64 once they are held in four bits."""
    g = v.reshape(*v.shape[:-1], -1, 32)
    f, p = torch.frexp(g.abs().amax(-1, keepdim=True))
    e = torch.where(f < 0.875, p - 3, p - 2).double().clamp(-125, 125)
    r = g.abs() / torch.pow(2.0, e)
    step = torch.where(r < 2, 0.5, torch.where(r < 4, 1.0, 2.0)).double()
    r = (torch.round(r / step) * step).clamp_max(6)
    return (torch.sign(g) * r * torch.pow(2.0, e)).reshape(v.shape)


def exact(case, seed):
    s = prepare(case, seed)
    if case["op"] == "linear":
        y = torch.addmm(s["b"].double(), s["x"].double(), _exact_values(s["codes"], s["scales"]).t())
        gate = {"none": lambda v: 1.0, "relu": lambda v: (v > 0).double(), "gelu": lambda v: torch.special.ndtr(v),
                "quick_gelu": lambda v: torch.sigmoid(1.702 * v), "silu": torch.sigmoid}[case["act"]]
        y *= gate(y)
        return y if s["r"] is None else y + s["r"].double()
    if case["op"] == "store":
        out = []
        for x in (s["k"], s["v"]):
            y = _exact_rounded(x.double())
            for b, n in enumerate(_counts(case)):
                y[b, n:] = 0
            out.append(y)
        return tuple(out)
    B, Tq, Hq, Hk, D = (case[k] for k in ("B", "Tq", "Hq", "Hk", "D"))
    G = Hq // Hk
    out = torch.zeros(B, Tq, Hq, D, dtype=torch.float64, device=DEVICE)
    for b, (n, t) in enumerate(zip(_lengths(case), _query_lengths(case))):
        if n == 0:
            continue
        pages = s["table"][b, :(n + case["page"] - 1) // case["page"]].long()
        hide = None
        if case["causal"]:
            hide = torch.ones(t, n, dtype=torch.bool, device=DEVICE).triu(n - t + 1)
        for h in range(Hk):
            k, v = (_exact_values(s["codes"][pages, i, h], s["scales"][pages, i, h]).reshape(-1, D)[:n]
                    for i in range(2))
            score = torch.tensordot(s["q"][b, :t, h * G:(h + 1) * G].double(), k, dims=([2], [1])) / math.sqrt(D)
            if hide is not None:
                score.masked_fill_(hide[:, None], -math.inf)
            out[b, :t, h * G:(h + 1) * G] = torch.tensordot(torch.softmax(score, -1), v, dims=([2], [0]))
    return out
