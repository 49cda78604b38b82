"""The token operators as they are measured: cases, inputs, plain forms and exact values.

Three operators of the transformer blocks that run over image tokens and
prompt rows: `linear` (matrix product with bias, activation and residual in
its epilogue), `qk_norm_rope` (head norm and position rotation with several
axes, in one pass) and `prefix_attention` (attention of a batch that shares
one long prefix). With `own` false, run() computes them in elementary torch
operations in 32 bits; with `own` true it makes the package's calls.
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
        # the prompted rows of a few crops through the first feed-forward layer
        dict(name="linear_prompt_rows", op="linear", M=37, K=1024, N=4096, act="gelu", residual=False, out="bf16"),
        # the prompted rows of the long-tail batch through an output projection, float32 residual stream
        dict(name="linear_longtail_rows", op="linear", M=19706, K=1024, N=1024, act="none", residual=True, out="f32"),
        # every token of 64 crops (24 x 24 each) through the first feed-forward layer
        dict(name="linear_image_tokens", op="linear", M=36864, K=1024, N=4096, act="gelu", residual=False, out="bf16"),
        # the newest token of eight sequences, grouped heads
        dict(name="rope_new_tokens", op="rope", B=8, T=1, Hq=32, Hk=8, D=128, rot=128, axes=1, norm=True,
             interleaved=False, dtype="bf16"),
        # partial rotation with pairs side by side, float32, odd sizes
        dict(name="rope_partial_f32", op="rope", B=3, T=1001, Hq=6, Hk=2, D=96, rot=64, axes=2, norm=True,
             interleaved=True, dtype="f32"),
        # 64 crops of 24 x 24 tokens behind 5 leading tokens, two axes, no norm
        dict(name="rope_image_tokens", op="rope", B=64, T=581, Hq=16, Hk=16, D=64, rot=64, axes=2, norm=False,
             interleaved=False, dtype="bf16"),
        # two clips of 8 frames of 48 x 48 tokens: time, height and width
        dict(name="rope_video", op="rope", B=2, T=18432, Hq=32, Hk=8, D=128, rot=128, axes=3, norm=True,
             interleaved=False, dtype="bf16"),
        # one prompt row against one image's tokens: latency
        dict(name="attend_one_row", op="attend", B=1, Tq=1, Hq=16, Hk=16, D=64, P=576, S=80, causal=False, ragged=False),
        # 37 prompt sets of up to 80 rows (padded, masked) against the 48 x 48 tokens of one image
        dict(name="attend_prompt_sets", op="attend", B=37, Tq=80, Hq=16, Hk=16, D=64, P=2304, S=80, causal=False,
             ragged=True),
        # a decoding step of 48 sequences with caches of their own behind a long shared prefix
        dict(name="attend_decode", op="attend", B=48, Tq=1, Hq=32, Hk=8, D=128, P=32768, S=1024, causal=True,
             ragged=True),
        # the first pass over eight requests behind a shared prefix
        dict(name="attend_prefill", op="attend", B=8, Tq=1024, Hq=32, Hk=8, D=128, P=8192, S=1024, causal=True,
             ragged=False),
    ]


def _spread(rng, low, high):
    """A whole number of low .. high, spread over its logarithm."""
    return max(low, min(high, int(round(math.exp(rng.uniform(math.log(low), math.log(high)))))))


def draw(rng):
    op = rng.choice(("linear", "rope", "attend"))
    if op == "linear":
        # tokens from one to a large batch; widths in whole 16-byte pieces, now and then not
        K = 8 * _spread(rng, 8, 512) if rng.random() < 0.85 else _spread(rng, 33, 2000)
        N = _spread(rng, 16, 4096)
        M = _spread(rng, 1, min(36864, 36864 * 1024 * 4096 // (K * N)))
        return dict(op=op, M=M, K=K, N=N, act=rng.choice(("none", "relu", "gelu", "quick_gelu", "silu")),
                    residual=rng.random() < 0.5, out=rng.choice(("bf16", "bf16", "f32")))
    if op == "rope":
        D = rng.choice((64, 64, 128, 128, 96, 80, 256))
        rot = D if rng.random() < 0.7 else 2 * rng.randint(4, D // 2)
        Hk = _spread(rng, 1, 16)
        Hq = Hk * rng.choice((1, 1, 2, 4, 5))
        B = _spread(rng, 1, 64)
        dtype = rng.choice(("bf16", "bf16", "f32"))
        most = 2 * 18432 * 40 * 128 // ((Hq + Hk) * D * (2 if dtype == "f32" else 1))
        return dict(op=op, B=B, T=_spread(rng, 1, max(1, min(30000, most // B))), Hq=Hq, Hk=Hk, D=D, rot=rot,
                    axes=rng.choice((1, 2, 3)), norm=rng.random() < 0.6, interleaved=rng.random() < 0.3, dtype=dtype)
    D = rng.choice((64, 128))
    Hk = _spread(rng, 1, 16)
    Hq = Hk * rng.choice((1, 2, 4, 7, 8))
    B = _spread(rng, 1, 64)
    P = _spread(rng, 1, 65536)
    Tq = 1 if rng.random() < 0.4 else _spread(rng, 2, 1024)
    S = max(Tq, _spread(rng, 16, 2048))
    # no more score values than the largest listed case has
    while B * Tq * Hq * (P + S) * D > 8 * 1024 * 32 * 9216 * 128:
        B, P, Tq = max(1, B * 3 // 4), max(1, P * 3 // 4), max(1, Tq * 3 // 4)
    return dict(op=op, B=B, Tq=Tq, Hq=Hq, Hk=Hk, D=D, P=P, S=S, causal=rng.random() < 0.6, ragged=rng.random() < 0.7)


def _own_lengths(case):
    """Own keys of each sequence, at least its queries: from half the space to all of it."""
    if not case["ragged"]:
        return [case["S"]] * case["B"]
    low = max(case["Tq"], case["S"] // 2)
    return [low + (7919 * (b + 1)) % (case["S"] - low + 1) for b in range(case["B"])]


def _query_lengths(case):
    """Rows in use of each sequence: all in decoding and causal passes, a padded batch otherwise."""
    if case["causal"] or not case["ragged"]:
        return [case["Tq"]] * case["B"]
    return [1 + (104729 * (b + 1)) % case["Tq"] for b in range(case["B"])]


def prepare(case, seed):
    g = torch.Generator(device=DEVICE)
    g.manual_seed(seed)

    def randn(*shape, scale=1.0, dtype=torch.bfloat16):
        return (torch.randn(*shape, generator=g, device=DEVICE) * scale).to(dtype)

    s = dict(case)
    if case["op"] == "linear":
        M, K, N = case["M"], case["K"], case["N"]
        s["x"] = randn(M, K)
        s["w"] = randn(N, K, scale=K ** -0.5)
        s["b"] = randn(N, scale=0.1)
        s["r"] = randn(M, N, dtype=TYPES[case["out"]]) if case["residual"] else None
    elif case["op"] == "rope":
        B, T, Hq, Hk, D, A = (case[k] for k in ("B", "T", "Hq", "Hk", "D", "axes"))
        dtype = TYPES[case["dtype"]]
        rows = randn(B, T, (Hq + Hk) * D, dtype=dtype)  # one projection's rows: queries, then keys
        s["q"] = rows[..., :Hq * D].unflatten(2, (Hq, D))
        s["k"] = rows[..., Hq * D:].unflatten(2, (Hk, D))
        s["gq"] = (1 + 0.1 * randn(D, dtype=torch.float32)).to(dtype) if case["norm"] else None
        s["gk"] = (1 + 0.1 * randn(D, dtype=torch.float32)).to(dtype) if case["norm"] else None
        # whole-number positions per axis, far ones among them; each frequency belongs to one axis
        span = torch.tensor([100000, 4096, 4096][:A] if A > 1 else [1000000], device=DEVICE)
        s["pos"] = (torch.rand(B, T, A, generator=g, device=DEVICE) * span).floor()
        half = case["rot"] // 2
        i = torch.arange(half, device=DEVICE)
        base = torch.exp(-math.log(10000.0) * i / half)
        s["freqs"] = torch.where(i % A == torch.arange(A, device=DEVICE)[:, None], base, 0.0).float().contiguous()
    else:
        B, Tq, Hq, Hk, D, P, S = (case[k] for k in ("B", "Tq", "Hq", "Hk", "D", "P", "S"))
        s["q"] = randn(B, Tq, Hq, D)
        kv = randn(P, 2, Hk, D)
        s["kp"], s["vp"] = kv[:, 0], kv[:, 1]
        kv = randn(B, S, 2, Hk, D)
        s["ko"], s["vo"] = kv[:, :, 0], kv[:, :, 1]
        s["own_len"] = torch.tensor(_own_lengths(case), dtype=torch.int32, device=DEVICE)
        s["q_len"] = torch.tensor(_query_lengths(case), dtype=torch.int32, device=DEVICE)
        s["mask"] = None
        if not case["causal"]:  # prompt rows: some of them hold no prompt
            s["mask"] = (torch.rand(B, S, generator=g, device=DEVICE) < 0.8).to(torch.uint8)
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
    y = torch.matmul(s["x"].float(), s["w"].float().t()) + s["b"].float()
    y = _act(y, s["act"])
    if s["r"] is not None:
        y = y + s["r"].float()
    return y.to(TYPES[s["out"]])


def _rotated(x, gain, cos, sin, s):
    u = x.float()
    if gain is not None:
        u = u / torch.sqrt((u * u).mean(-1, keepdim=True) + 1e-6) * gain.float()
    half = s["rot"] // 2
    y = u.clone()
    if s["interleaved"]:
        a, b = u[..., 0:s["rot"]:2], u[..., 1:s["rot"]:2]
        y[..., 0:s["rot"]:2] = a * cos - b * sin
        y[..., 1:s["rot"]:2] = b * cos + a * sin
    else:
        a, b = u[..., :half], u[..., half:s["rot"]]
        y[..., :half] = a * cos - b * sin
        y[..., half:s["rot"]] = b * cos + a * sin
    return y.to(x.dtype)


def _rope(s):
    angle = (s["pos"].double()[..., None] * s["freqs"].double()).sum(-2)[:, :, None]
    cos, sin = torch.cos(angle).float(), torch.sin(angle).float()
    return _rotated(s["q"], s["gq"], cos, sin, s), _rotated(s["k"], s["gk"], cos, sin, s)


def _attend(s):
    B, Tq, Hq, Hk, D, P, S = (s[k] for k in ("B", "Tq", "Hq", "Hk", "D", "P", "S"))
    G = Hq // Hk
    q = s["q"].float().reshape(B, Tq, Hk, G, D).permute(0, 2, 1, 3, 4) * D ** -0.5  # [B, Hk, Tq, G, D]
    qs = q.permute(1, 0, 2, 3, 4).reshape(Hk, B * Tq * G, D)
    kp, vp = (s[n].float().permute(1, 0, 2) for n in ("kp", "vp"))                  # [Hk, P, D]
    ko, vo = (s[n].float().permute(0, 2, 1, 3) for n in ("ko", "vo"))               # [B, Hk, S, D]
    shared = torch.matmul(qs, kp.transpose(1, 2)).reshape(Hk, B, Tq * G, P)
    mine = torch.matmul(q.reshape(B, Hk, Tq * G, D), ko.transpose(2, 3)).transpose(0, 1)  # [Hk, B, Tq G, S]
    j = torch.arange(S, device=mine.device)
    n = s["own_len"].long()
    seen = (j < n[:, None])[:, None]                                                # [B, 1, S]
    if s["mask"] is not None:
        seen = seen & (s["mask"] != 0)[:, None]
    if s["causal"]:
        t = torch.arange(Tq, device=mine.device).repeat_interleave(G)
        seen = seen & (j <= (n - s["q_len"])[:, None, None] + t[:, None])
    mine = torch.where(seen, mine, -math.inf)
    top = torch.maximum(shared.amax(-1, keepdim=True), mine.amax(-1, keepdim=True))
    shared, mine = torch.exp(shared - top), torch.exp(mine - top)
    total = shared.sum(-1, keepdim=True) + mine.sum(-1, keepdim=True)
    y = torch.matmul(shared.reshape(Hk, B * Tq * G, P), vp).reshape(Hk, B, Tq * G, D)
    y = y + torch.matmul(mine.transpose(0, 1), vo).transpose(0, 1)
    y = (y / total).reshape(Hk, B, Tq, G, D).permute(1, 2, 0, 3, 4).reshape(B, Tq, Hq, D)
    used = torch.arange(Tq, device=y.device) < s["q_len"][:, None]
    return torch.where(used[..., None, None], y, 0.0).to(torch.bfloat16)


def run(state):
    s = state
    if own:
        import prompt_conditioned_keypoint_amd as gkd
        if s["op"] == "linear":
            return gkd.linear(s["x"], s["w"], bias=s["b"], residual=s["r"], act=s["act"], out_dtype=TYPES[s["out"]])
        if s["op"] == "rope":
            return gkd.qk_norm_rope(s["q"], s["k"], s["pos"], s["freqs"], q_weight=s["gq"], k_weight=s["gk"], eps=1e-6,
                                    interleaved=s["interleaved"])
        return gkd.prefix_attention(s["q"], s["kp"], s["vp"], s["ko"], s["vo"], own_len=s["own_len"], q_len=s["q_len"],
                                    own_mask=s["mask"], causal=s["causal"], out=s["out"])
    return {"linear": _linear, "rope": _rope, "attend": _attend}[s["op"]](s)


def work(case):
    c = case
    if c["op"] == "linear":
        e = 4 if c["out"] == "f32" else 2
        moved = 2 * (c["M"] * c["K"] + c["N"] * c["K"] + c["N"]) + e * c["M"] * c["N"] * (2 if c["residual"] else 1)
        return {"bytes": moved, "flops": 2 * c["M"] * c["N"] * c["K"]}
    if c["op"] == "rope":
        n = c["B"] * c["T"] * (c["Hq"] + c["Hk"]) * c["D"]
        e = 4 if c["dtype"] == "f32" else 2
        return {"bytes": 2 * e * n + 4 * c["B"] * c["T"] * c["axes"], "flops": (7 if c["norm"] else 3) * n}
    rows, keys, pairs = 0, 0, 0
    for n, t in zip(_own_lengths(c), _query_lengths(c)):
        rows += t
        keys += n
        pairs += t * c["P"] + (t * (n - t) + t * (t + 1) // 2 if c["causal"] else t * n)
    moved = 4 * rows * c["Hq"] * c["D"] + 4 * (c["P"] + keys) * c["Hk"] * c["D"]
    return {"bytes": moved, "flops": 4 * pairs * c["Hq"] * c["D"]}


def exact(case, seed):
    s = prepare(case, seed)
    if case["op"] == "linear":
        y = torch.addmm(s["b"].double(), s["x"].double(), s["w"].double().t())
        gate = {"none": lambda v: 1.0, "relu": lambda v: (v > 0).double(), "gelu": lambda v: torch.special.ndtr(v),
                "quick_gelu": lambda v: torch.sigmoid(1.702 * v), "silu": torch.sigmoid}[case["act"]]
        y *= gate(y)
        return y if s["r"] is None else y + s["r"].double()
    if case["op"] == "rope":
        out = []
        half = case["rot"] // 2
        # the rotation as a product with exp(i phi); phi summed axis by axis
        phi = sum(s["pos"][..., a:a + 1].double() * s["freqs"][a].double() for a in range(case["axes"]))
        turn = torch.polar(torch.ones_like(phi), phi).unsqueeze(2)
        for x, gain in ((s["q"], s["gq"]), (s["k"], s["gk"])):
            u = x.double()
            if gain is not None:
                u = u * (u.pow(2).mean(-1, keepdim=True) + 1e-6).rsqrt() * gain.double()
            r, rest = u[..., :case["rot"]], u[..., case["rot"]:]
            r = r.unflatten(-1, (half, 2) if case["interleaved"] else (2, half))
            if not case["interleaved"]:
                r = r.transpose(-1, -2)
            r = torch.view_as_real(torch.view_as_complex(r.contiguous()) * turn)
            if not case["interleaved"]:
                r = r.transpose(-1, -2)
            out.append(torch.cat([r.flatten(-2), rest], -1))
        return tuple(out)
    B, Tq, Hq, Hk, D, P, S = (case[k] for k in ("B", "Tq", "Hq", "Hk", "D", "P", "S"))
    out = torch.zeros(B, Tq, Hq, D, dtype=torch.float64, device=DEVICE)
    for b, (n, t) in enumerate(zip(_own_lengths(case), _query_lengths(case))):
        hide = torch.zeros(t, n, dtype=torch.bool, device=DEVICE)
        if s["mask"] is not None:
            hide |= s["mask"][b, :n] == 0
        if case["causal"]:
            hide |= torch.ones(t, n, dtype=torch.bool, device=DEVICE).triu(n - t + 1)
        for h in range(Hk):
            g = slice(h * (Hq // Hk), (h + 1) * (Hq // Hk))
            k = torch.cat([s["kp"][:, h], s["ko"][b, :n, h]]).double()
            v = torch.cat([s["vp"][:, h], s["vo"][b, :n, h]]).double()
            score = torch.tensordot(s["q"][b, :t, g].double(), k, dims=([2], [1])) / math.sqrt(D)
            score[..., P:].masked_fill_(hide[:, None], -math.inf)
            out[b, :t, g] = torch.tensordot(torch.softmax(score, -1), v, dims=([2], [0]))
    return out
