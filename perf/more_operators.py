"""Operators of attention blocks and image blocks as they are measured: cases, inputs,
plain forms.

  attn        attention: the forward alone (a prefill, one token over a cache) or a
              training pass, forward and the backward that recomputes the probabilities
  rotary      rotary positions with several axes (time, height, width) on q and k
  group_norm  group norm with an activation, channels last: inference, or forward and
              backward

run() computes the plain form in elementary torch operations (float32, rounded once at
the end; angles in float64), or, with `own` set, calls the library's entry points.
exact() computes the same from the definitions in float64.
"""
import math

import torch

own = False

DTYPES = {"f32": torch.float32, "bf16": torch.bfloat16, "f16": torch.float16}
BYTES = {"f32": 4, "bf16": 2, "f16": 2}


# ---------------------------------------------------------------------------
# cases
#
# attn: B sequences of up to Sq queries and Sk keys, H query and KV key heads of D.
# right 0 is causal, -1 unbounded; left likewise.  lens: "full" (every sequence the whole
# length), "padded" (lengths of a padded batch), "packed" (sequences one behind another).
# rotary: sections are the numbers of pairs that turn by each axis.

def listed():
    return [
        # a long prompt, grouped heads
        dict(name="attn_prefill_bf16", op="attn", train=False, B=2, Sq=8192, Sk=8192, H=32, KV=8,
             D=128, left=-1, right=0, lens="full", dtype="bf16"),
        # one generated token for each of 8 requests, caches of up to 32768 tokens
        dict(name="attn_token_bf16", op="attn", train=False, B=8, Sq=1, Sk=32768, H=32, KV=8,
             D=128, left=-1, right=0, lens="padded", dtype="bf16"),
        # one token, a short cache: latency
        dict(name="attn_token_short_f16", op="attn", train=False, B=1, Sq=1, Sk=517, H=8, KV=8,
             D=64, left=-1, right=0, lens="full", dtype="f16"),
        # a training step of a causal model
        dict(name="attn_train_bf16", op="attn", train=True, B=2, Sq=4096, Sk=4096, H=32, KV=8,
             D=128, left=-1, right=0, lens="full", dtype="bf16"),
        # documents of a training batch packed one behind another
        dict(name="attn_packed_f16", op="attn", train=True, B=13, Sq=2048, Sk=2048, H=16, KV=16,
             D=64, left=-1, right=0, lens="packed", dtype="f16"),
        # image tokens in full precision, odd in every extent, a window around each
        dict(name="attn_window_f32", op="attn", train=True, B=2, Sq=1027, Sk=777, H=6, KV=3,
             D=72, left=255, right=130, lens="padded", dtype="f32"),
        # q and k of a video: (frame, row, column) positions, frequencies of each axis its own
        dict(name="rotary_video_bf16", op="rotary", B=2, S=11880, H=24, KV=8, D=128,
             sections="16 24 24", interleaved=False, positions="int", inverse=False,
             dtype="bf16"),
        # one token of each of 48 requests at far positions
        dict(name="rotary_token_f16", op="rotary", B=48, S=1, H=32, KV=8, D=128, sections="64",
             interleaved=True, positions="int", inverse=False, dtype="f16"),
        # image patches at fractional positions, part of each head turned, the backward
        dict(name="rotary_image_f32", op="rotary", B=3, S=1369, H=12, KV=12, D=72,
             sections="15 15", interleaved=False, positions="float", inverse=True, dtype="f32"),
        # a decoder's wide map, training
        dict(name="gn_decoder_bf16", op="group_norm", train=True, N=8, H=128, W=128, C=512, G=32,
             act="silu", dtype="bf16"),
        # an odd map and odd groups, training
        dict(name="gn_odd_f32", op="group_norm", train=True, N=3, H=37, W=29, C=150, G=10,
             act="leaky_relu", dtype="f32"),
        # a small map in inference: latency
        dict(name="gn_small_f16", op="group_norm", train=False, N=1, H=16, W=16, C=640, G=32,
             act="silu", dtype="f16"),
    ]


def _log_int(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(("attn", "attn", "rotary", "group_norm"))
    dtype = rng.choice(("bf16", "bf16", "f16", "f32"))
    if op == "group_norm":
        G = rng.choice((1, 4, 8, 16, 32))
        C = G * _log_int(rng, 1, 1024 // G)
        H, W = _log_int(rng, 1, 256), _log_int(rng, 1, 256)
        N = max(1, min(_log_int(rng, 1, 16), (60 << 20) // (H * W * C)))
        return dict(op=op, train=rng.random() < 0.7, N=N, H=H, W=W, C=C, G=G,
                    act=rng.choice(("identity", "silu", "gelu", "leaky_relu")), dtype=dtype)
    B = _log_int(rng, 1, 32)
    KV = rng.choice((1, 2, 3, 4, 8))
    H = KV * rng.choice((1, 1, 2, 4, 5, 8))
    D = rng.choice((32, 40, 64, 64, 72, 80, 96, 128, 128, 128))
    if op == "rotary":
        pairs = rng.choice((D // 2, D // 2, D // 4))
        axes = rng.choice((1, 2, 3))
        cut = sorted(rng.sample(range(1, pairs), axes - 1))
        S = max(1, min(_log_int(rng, 1, 16384), (60 << 20) // (B * (H + KV) * D)))
        return dict(op=op, B=B, S=S, H=H, KV=KV, D=D,
                    sections=" ".join(str(b - a) for a, b in zip([0] + cut, cut + [pairs])),
                    interleaved=rng.random() < 0.5, positions=rng.choice(("int", "float")),
                    inverse=rng.random() < 0.5, dtype=dtype)
    train = rng.random() < 0.5
    lens = rng.choice(("full", "padded", "packed"))
    Sk = _log_int(rng, 1, 8192)
    Sq = Sk if lens == "packed" or rng.random() < 0.4 else _log_int(rng, 1, 8192)
    if not train and lens != "packed" and rng.random() < 0.4:
        Sq, Sk = rng.choice((1, 1, 1, 2, 5)), _log_int(rng, 64, 32768)
    # products in float32 cost about ten times those in 16 bits
    most = 2 ** 33 if dtype != "f32" else 2 ** 30
    B = max(1, min(B, most // (Sq * Sk * H), (1 << 28) // (max(Sq, Sk) * H * D)))
    while Sq * Sk * H * B > most and Sq > 1:
        Sq, Sk = Sq // 2, max(1, Sk // 2)
        Sq = Sk if lens == "packed" else Sq
    right = rng.choice((0, 0, -1, _log_int(rng, 1, 1024)))
    return dict(op=op, train=train, B=B, Sq=Sq, Sk=Sk, H=H, KV=KV, D=D,
                left=rng.choice((-1, -1, _log_int(rng, 1, 1024))), right=right, lens=lens,
                dtype=dtype)


def _sections(c):
    return [int(n) for n in c["sections"].split()]


def _lengths(c):
    """(queries, keys) of each sequence, two lists: the same for every seed."""
    B, Sq, Sk = c["B"], c["Sq"], c["Sk"]
    if c["lens"] == "full":
        return [Sq] * B, [Sk] * B
    # the first is whole, the others spread over (0, 1) of it without a pattern
    part = [1.0] + [(b * 0.61803398875) % 1.0 for b in range(1, B)]
    k = [max(1, math.ceil(p * Sk)) for p in part]
    if c["lens"] == "packed":
        return list(k), k
    return [max(1, math.ceil(part[-b] * Sq)) for b in range(B)], k


def _pairs(c):
    """Visible (query, key) pairs of all sequences."""
    n = 0
    for lq, lk in zip(*_lengths(c)):
        i = torch.arange(lq, dtype=torch.int64) + (lk - lq)
        lo = (i - c["left"]).clamp(min=0) if c["left"] >= 0 else torch.zeros_like(i)
        hi = (i + c["right"] + 1).clamp(max=lk) if c["right"] >= 0 else torch.full_like(i, lk)
        n += int((hi - lo).clamp(min=0).sum())
    return n


def work(c):
    e = BYTES[c["dtype"]]
    if c["op"] == "group_norm":
        n = c["N"] * c["H"] * c["W"] * c["C"]
        # forward: x, y; backward: x, dy, dx
        return {"bytes": n * e * (5 if c["train"] else 2), "flops": n * (40 if c["train"] else 15)}
    if c["op"] == "rotary":
        n = c["B"] * c["S"] * (c["H"] + c["KV"]) * c["D"]
        return {"bytes": 2 * n * e + c["B"] * c["S"] * 4 * len(_sections(c)), "flops": 3 * n}
    lq, lk = _lengths(c)
    q, kv = sum(lq) * c["H"] * c["D"] * e, 2 * sum(lk) * c["KV"] * c["D"] * e
    flops = (14.0 if c["train"] else 4.0) * c["D"] * c["H"] * _pairs(c)
    if not c["train"]:
        return {"bytes": 2 * q + kv, "flops": flops}
    # forward: q, k, v, out, lse; backward: those, dout, and the three gradients
    return {"bytes": 6 * q + 3 * kv + 8 * sum(lq) * c["H"], "flops": flops}


# ---------------------------------------------------------------------------
# inputs

def _normal(gen, *shape):
    return torch.randn(*shape, generator=gen, device="cuda")


def _starts(lens):
    return torch.tensor([0] + lens, dtype=torch.int32).cumsum(0, dtype=torch.int32).cuda()


def _prepare_attn(c, s, gen, dt):
    B, H, KV, D = c["B"], c["H"], c["KV"], c["D"]
    lq, lk = _lengths(c)
    s["lq"], s["lk"] = lq, lk
    s["causal"], s["window"] = c["right"] == 0 and c["left"] < 0, (c["left"], c["right"])
    if c["lens"] == "packed":
        lead = (sum(lq),)
        s["q_starts"], s["k_starts"] = _starts(lq), _starts(lk)
        # the gather of a padded batch from the packed rows and back, for the plain form
        n = torch.arange(c["Sq"], device="cuda")
        s["held"] = n[None] < torch.tensor(lq, device="cuda")[:, None]
        s["rows"] = torch.where(s["held"], s["q_starts"][:-1, None].long() + n, 0)
    else:
        lead = (B, c["Sq"])
        if c["lens"] == "padded":
            s["q_lens"] = torch.tensor(lq, dtype=torch.int32, device="cuda")
            s["k_lens"] = torch.tensor(lk, dtype=torch.int32, device="cuda")
    if c["lens"] == "packed" or (c["lens"] == "full" and c["Sq"] == c["Sk"]):
        # slices of one projection
        qkv = _normal(gen, *lead, H + 2 * KV, D).to(dt)
        s["q"], s["k"], s["v"] = qkv.split((H, KV, KV), -2)
    else:
        s["q"] = _normal(gen, *lead, H, D).to(dt)
        s["k"] = _normal(gen, B, c["Sk"], KV, D).to(dt)
        s["v"] = _normal(gen, B, c["Sk"], KV, D).to(dt)
    if c["train"]:
        s["dout"] = _normal(gen, *lead, H, D).to(dt)


def _prepare_rotary(c, s, gen, dt):
    B, S, H, KV, D = c["B"], c["S"], c["H"], c["KV"], c["D"]
    qkv = _normal(gen, B, S, H + 2 * KV, D).to(dt)
    s["q"], s["k"], _ = qkv.split((H, KV, KV), -2)
    sections = _sections(c)
    axes, pairs = len(sections), sum(sections)
    far = 1 << 20 if S == 1 else 4 * S
    if c["positions"] == "int":
        s["positions"] = torch.randint(0, far, (B, S, axes), generator=gen, device="cuda",
                                       dtype=torch.int32)
    else:
        s["positions"] = 64 * torch.rand(B, S, axes, generator=gen, device="cuda") - 32
    ramps = [torch.arange(n, dtype=torch.float64) / n for n in sections]
    s["inv_freq"] = (10000.0 ** -torch.cat(ramps)).cuda()
    s["axis"] = torch.repeat_interleave(torch.arange(axes, dtype=torch.int32),
                                        torch.tensor(sections)).cuda()
    s["pairs"], s["axes"] = pairs, axes


def _prepare_group_norm(c, s, gen, dt):
    N, H, W, C = c["N"], c["H"], c["W"], c["C"]
    # channels of their own mean and size
    x = _normal(gen, N, H, W, C) * (0.5 + torch.rand(C, generator=gen, device="cuda"))
    s["x"] = x.add_(0.5 * _normal(gen, C)).to(dt)
    s["weight"], s["bias"] = 1 + 0.2 * _normal(gen, C), 0.1 * _normal(gen, C)
    s["eps"], s["slope"] = 1e-5, 0.01
    if c["train"]:
        s["dy"] = (0.01 * _normal(gen, N, H, W, C)).to(dt)


def prepare(c, seed):
    gen = torch.Generator(device="cuda").manual_seed(seed)
    dt = DTYPES[c["dtype"]]
    s = dict(c, dt=dt)
    {"attn": _prepare_attn, "rotary": _prepare_rotary,
     "group_norm": _prepare_group_norm}[c["op"]](c, s, gen, dt)
    return s


# ---------------------------------------------------------------------------
# plain forms

def _visible(s):
    """[B, Sq, Sk]: which keys each query sees."""
    lq = torch.tensor(s["lq"], device="cuda")[:, None, None]
    lk = torch.tensor(s["lk"], device="cuda")[:, None, None]
    i = torch.arange(s["Sq"], device="cuda")[None, :, None]
    j = torch.arange(s["Sk"], device="cuda")[None, None, :]
    see = (i < lq) & (j < lk)
    at = i + (lk - lq)
    if s["left"] >= 0:
        see = see & (j >= at - s["left"])
    if s["right"] >= 0:
        see = see & (j <= at + s["right"])
    return see


def _plain_attn(s):
    B, Sq, Sk, H, KV, D = (s[k] for k in ("B", "Sq", "Sk", "H", "KV", "D"))
    G, scale = H // KV, 1 / math.sqrt(D)
    packed = s["lens"] == "packed"
    names = ("q", "k", "v") + (("dout",) if s["train"] else ())
    see = _visible(s)[:, None]
    new = lambda t: torch.empty_like(t, memory_format=torch.contiguous_format)  # noqa: E731
    out = dict(out=new(s["q"]))
    if s["train"]:
        out.update(dq=new(s["q"]), dk=new(s["k"]), dv=new(s["v"]))
    # as many key heads at a time as their scores take 2 GiB
    step = max(1, min(KV, (1 << 29) // max(1, B * G * Sq * Sk)))
    for h in range(0, KV, step):
        n = min(step, KV - h)

        def heads(name):                     # [B, n, rows, D], queries as [B, n, G * Sq, D]
            m = G if name in ("q", "dout") else 1
            t = s[name][..., h * m:(h + n) * m, :].float()
            if packed:
                t = t[s["rows"]] * s["held"][..., None, None]
            t = t.transpose(1, 2).contiguous()
            return t.reshape(B, n, m * t.shape[2], D)

        def put(name, t, m):                 # back into the heads' places
            t = t.reshape(B, n * m, -1, D).transpose(1, 2)
            if packed:
                t = t[s["held"]]
            out[name][..., h * m:(h + n) * m, :] = t.to(s["dt"])

        x = {name: heads(name) for name in names}
        p = x["q"] @ x["k"].transpose(2, 3).contiguous()
        p = (p * scale).view(B, n * G, Sq, Sk).masked_fill_(~see, -math.inf)
        m = p.amax(-1, keepdim=True)
        p = torch.exp(p - torch.where(m == -math.inf, 0.0, m))
        total = p.sum(-1, keepdim=True)
        p = (p / torch.where(total == 0, 1.0, total)).view(B, n, G * Sq, Sk)
        o = p @ x["v"]
        put("out", o, G)
        if s["train"]:
            do = x["dout"]
            put("dv", p.transpose(2, 3).contiguous() @ do, 1)
            ds = do @ x["v"].transpose(2, 3).contiguous()
            ds = p * (ds - (do * o).sum(-1, keepdim=True)) * scale
            put("dq", ds @ x["k"], G)
            put("dk", ds.transpose(2, 3).contiguous() @ x["q"], 1)
    return out


def _plain_rotary(s):
    angle = s["positions"].double()[..., s["axis"].long()] * s["inv_freq"]
    if s["inverse"]:
        angle = -angle
    co, si = torch.cos(angle).float()[:, :, None], torch.sin(angle).float()[:, :, None]
    out, n = {}, s["pairs"]
    for name in ("q", "k"):
        x = s[name].float()
        if s["interleaved"]:
            a, b = x[..., 0:2 * n:2], x[..., 1:2 * n:2]
            turned = torch.stack((a * co - b * si, b * co + a * si), -1).flatten(-2)
        else:
            a, b = x[..., :n], x[..., n:2 * n]
            turned = torch.cat((a * co - b * si, b * co + a * si), -1)
        out[name] = torch.cat((turned, x[..., 2 * n:]), -1).to(s["dt"])
    return out


def _act(z, s):
    """act(z) and act'(z)."""
    if s["act"] == "identity":
        return z, torch.ones_like(z)
    if s["act"] == "leaky_relu":
        slope = torch.where(z >= 0, 1.0, s["slope"])
        return z * slope, slope
    if s["act"] == "silu":
        sg = 1 / (1 + torch.exp(-z))
        return z * sg, sg * (1 + z * (1 - sg))
    cdf = 0.5 * (1 + torch.erf(z * math.sqrt(0.5)))
    return z * cdf, cdf + z * torch.exp(-0.5 * z * z) * (1 / math.sqrt(2 * math.pi))


def _plain_group_norm(s):
    N, C, G = s["N"], s["C"], s["G"]
    x = s["x"].float().view(N, -1, G, C // G)
    x = x - x.mean((1, 3), keepdim=True)
    rstd = 1 / torch.sqrt((x * x).mean((1, 3), keepdim=True) + s["eps"])
    xhat = x * rstd
    w = s["weight"].view(G, C // G)
    y, slope = _act(xhat * w + s["bias"].view(G, C // G), s)
    out = dict(y=y.to(s["dt"]).view(s["x"].shape))
    if s["train"]:
        dz = s["dy"].float().view(x.shape) * slope
        out["dweight"] = (dz * xhat).sum((0, 1)).view(C)
        out["dbias"] = dz.sum((0, 1)).view(C)
        dz = dz * w
        dx = dz - dz.mean((1, 3), keepdim=True) - xhat * (dz * xhat).mean((1, 3), keepdim=True)
        out["dx"] = (dx * rstd).to(s["dt"]).view(s["x"].shape)
    return out


# ---------------------------------------------------------------------------
# the library's operators

def _own(s):
    import place_batchnorm_activation_amd as iabn
    new = lambda t: torch.empty_like(t, memory_format=torch.contiguous_format)  # noqa: E731
    if s["op"] == "attn":
        q, k, v = s["q"], s["k"], s["v"]
        spec = iabn.AttentionSpec(causal=s["causal"], window=s["window"])
        kw = {n: s[n] for n in ("q_starts", "k_starts", "q_lens", "k_lens") if n in s}
        if s["lens"] == "packed":
            kw.update(max_q=s["Sq"], max_k=s["Sk"])
        out = new(q)
        lse = iabn.attention_lse(q) if s["train"] else None
        iabn.iabn_attention_forward(spec, q, k, v, out, lse,
                                    iabn.attention_workspace(spec, q, k, **kw), **kw)
        if not s["train"]:
            return dict(out=out)
        dq, dk, dv = new(q), new(k), new(v)
        iabn.iabn_attention_backward(spec, q, k, v, out, lse, s["dout"], dq, dk, dv,
                                     iabn.attention_workspace(spec, q, k, backward=True, **kw),
                                     **kw)
        return dict(out=out, dq=dq, dk=dk, dv=dv)
    if s["op"] == "rotary":
        spec = iabn.RotarySpec(s["D"], inv_freq=s["inv_freq"], axis=s["axis"],
                               axes=s["axes"], interleaved=s["interleaved"])
        q, k = new(s["q"]), new(s["k"])
        iabn.iabn_rotary(spec, s["positions"], s["q"], q, s["k"], k, inverse=s["inverse"])
        return dict(q=q, k=k)
    x, w, b, G = s["x"], s["weight"], s["bias"], s["G"]
    y = torch.empty_like(x)
    ws = iabn.group_norm_workspace(x, G)
    args = dict(act=s["act"], act_param=s["slope"])
    if not s["train"]:
        iabn.iabn_group_norm_forward(x, y, G, w, b, ws, eps=s["eps"], **args)
        return dict(y=y)
    stats = torch.empty(s["N"], G, 2, device="cuda")
    iabn.iabn_group_norm_forward(x, y, G, w, b, ws, eps=s["eps"], stats=stats, **args)
    dx, dw, db = torch.empty_like(x), torch.empty_like(w), torch.empty_like(b)
    iabn.iabn_group_norm_backward(x, s["dy"], dx, G, w, b, stats, ws, dweight=dw, dbias=db, **args)
    return dict(y=y, dweight=dw, dbias=db, dx=dx)


def run(s):
    if own:
        return _own(s)
    return {"attn": _plain_attn, "rotary": _plain_rotary,
            "group_norm": _plain_group_norm}[s["op"]](s)


# ---------------------------------------------------------------------------
# the definitions in 64 bits

def _exact_attn(c, s):
    D, G = c["D"], c["H"] // c["KV"]
    names = ["out"] + (["dq", "dk", "dv"] if c["train"] else [])
    like = dict(out="q", dq="q", dk="k", dv="v")
    res = {n: torch.zeros(s[like[n]].shape, dtype=torch.float64, device="cuda") for n in names}
    qa = ka = 0
    for b, (lq, lk) in enumerate(zip(s["lq"], s["lk"])):
        if c["lens"] == "packed":
            rows, cols = (slice(qa, qa + lq),), (slice(ka, ka + lk),)
            qa, ka = qa + lq, ka + lk
        else:
            rows, cols = (b, slice(0, lq)), (b, slice(0, lk))
        away = torch.arange(lk, device="cuda") - torch.arange(lk - lq, lk, device="cuda")[:, None]
        hidden = torch.zeros(lq, lk, dtype=torch.bool, device="cuda")
        if c["left"] >= 0:
            hidden |= away < -c["left"]
        if c["right"] >= 0:
            hidden |= away > c["right"]
        empty = hidden.all(1)
        for h in range(c["H"]):
            q, k, v = s["q"][rows + (h,)].double(), s["k"][cols + (h // G,)].double(), \
                s["v"][cols + (h // G,)].double()
            logits = torch.mm(q, k.t().contiguous()).div_(D ** 0.5)
            logits[hidden] = -math.inf
            p = torch.softmax(logits, 1)
            p[empty] = 0.0
            o = torch.mm(p, v)
            res["out"][rows + (h,)] = o
            if c["train"]:
                do = s["dout"][rows + (h,)].double()
                res["dv"][cols + (h // G,)] += torch.mm(p.t().contiguous(), do)
                dp = torch.mm(do, v.t().contiguous())
                dl = p * dp
                dl -= p * dl.sum(1, keepdim=True)
                dl /= D ** 0.5
                res["dq"][rows + (h,)] = torch.mm(dl, k)
                res["dk"][cols + (h // G,)] += torch.mm(dl.t().contiguous(), q)
    return res


def _exact_rotary(c, s):
    """Each pair as a complex number, times e^(i angle)."""
    n = s["pairs"]
    where = s["positions"].double()
    angles = torch.cat([where[..., a:a + 1] * s["inv_freq"][s["axis"] == a]
                        for a in range(s["axes"])], -1)
    turn = torch.polar(torch.ones_like(angles), -angles if c["inverse"] else angles)[:, :, None]
    res = {}
    for name in ("q", "k"):
        x = s[name].double()
        y = x.clone()
        if c["interleaved"]:
            z = torch.view_as_complex(x[..., :2 * n].unflatten(-1, (n, 2)).contiguous()) * turn
            y[..., :2 * n] = torch.view_as_real(z).flatten(-2)
        else:
            z = torch.complex(x[..., :n].contiguous(), x[..., n:2 * n].contiguous()) * turn
            y[..., :n], y[..., n:2 * n] = z.real, z.imag
        res[name] = y
    return res


def _exact_group_norm(c, s):
    N, C, G = c["N"], c["C"], c["G"]
    flat = lambda t: t.double().reshape(N, -1, G, C // G).transpose(1, 2).flatten(2)  # noqa: E731
    back = lambda t: t.view(N, G, -1, C // G).transpose(1, 2).reshape(s["x"].shape)  # noqa: E731
    x = flat(s["x"])
    var, mean = torch.var_mean(x, -1, unbiased=False, keepdim=True)
    rstd = (var + s["eps"]).rsqrt()
    xhat = (x - mean) * rstd
    spread = lambda v: v.double().view(1, G, 1, -1).expand(N, G, x.shape[2] * G // C, C // G) \
        .flatten(2)  # noqa: E731
    w = spread(s["weight"])
    z = xhat * w + spread(s["bias"])
    if c["act"] == "identity":
        y, d = z, torch.ones_like(z)
    elif c["act"] == "leaky_relu":
        y, d = torch.where(z < 0, s["slope"] * z, z), torch.where(z < 0, s["slope"], 1.0)
    elif c["act"] == "silu":
        sg = torch.sigmoid(z)
        y, d = z * sg, sg + z * sg * torch.sigmoid(-z)
    else:
        phi = torch.special.ndtr(z)
        y, d = z * phi, phi + z * torch.exp(-z * z / 2) / (2 * math.pi) ** 0.5
    res = dict(y=back(y))
    if c["train"]:
        dz = flat(s["dy"]) * d
        channels = lambda t: t.view(N, G, -1, C // G).sum((0, 2)).view(C)  # noqa: E731
        res["dweight"], res["dbias"] = channels(dz * xhat), channels(dz)
        g = dz * w
        res["dx"] = back(rstd * (g - g.mean(-1, keepdim=True) -
                                 xhat * (g * xhat).mean(-1, keepdim=True)))
    return res


def exact(c, seed):
    s = prepare(c, seed)
    return {"attn": _exact_attn, "rotary": _exact_rotary,
            "group_norm": _exact_group_norm}[c["op"]](c, s)
