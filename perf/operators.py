"""Performance cases of the decoder-layer operators around the MoE layer.

Four operators make up the half of a decoder layer that is not the mixture of
experts: the residual addition with RMS norm (optionally to 8 bits), the position
rotation that appends keys and values to a paged cache, the attention of one new
token over that cache, and the matrix product with its epilogue.  Sizes follow the
MoE layer's workloads (hidden size 4096; 1, 8, 32 and 8192 tokens) with generic head
layouts.

`own` selects between the plain form (elementary torch operations in 32 bits) and
the library's entry points.
"""
import math

import torch

own = False

DT = {"bf16": torch.bfloat16, "f16": torch.float16, "f32": torch.float32, "e4m3": torch.float8_e4m3fn}
SIZE = {"bf16": 2, "f16": 2, "f32": 4, "e4m3": 1}
E4M3_MAX = 448.0
TINY = 2.0 ** -126
EPS = 1e-6

# No drawn case costs more than the largest listed one of its operator.
NORM_ELEMS = 8192 * 4096
APPEND_ELEMS = 8192 * 48 * 128
KV_BYTES = 64 * 12288 * 8 * 128 * 2
MM_FLOPS = 2 * 8192 * 6144 * 4096


def listed():
    return [
        # one decode token entering a layer's quantised projection
        dict(name="norm-decode-1", op="norm", T=1, H=4096, x="bf16", res="bf16", y="e4m3"),
        # an odd batch of rows of an odd width, residual stream kept in 32 bits
        dict(name="norm-ragged", op="norm", T=777, H=5003, x="f16", res="f32", y="f16"),
        # a prompt of 8192 tokens entering a quantised projection
        dict(name="norm-prompt-8192", op="norm", T=8192, H=4096, x="bf16", res="bf16", y="e4m3"),
        # a decode step of 8 sequences: one token each into pages of 16
        dict(name="append-decode-8", op="append", T=8, hq=32, hkv=8, D=128, page=16, x="bf16", kv="bf16", rot=128,
             interleaved=False),
        # a prompt of 8192 tokens into an 8-bit cache
        dict(name="append-prompt-8192", op="append", T=8192, hq=32, hkv=8, D=128, page=64, x="bf16", kv="e4m3",
             rot=128, interleaved=False),
        # one user's conversation: a single sequence, where the split over its length counts
        dict(name="attend-1x4097", op="attend", B=1, lo=4097, hi=4097, hq=32, hkv=8, D=128, page=16, q="bf16",
             kv="bf16", window=0),
        # a small model's short ragged batch: one key head per query head, 96-wide heads, a sliding window, and
        # sequences with no token yet
        dict(name="attend-window-ragged", op="attend", B=19, lo=0, hi=2500, hq=12, hkv=12, D=96, page=7, q="f16",
             kv="f16", window=1000),
        # a serving batch of 32 ragged sequences in a 16-bit cache
        dict(name="attend-32-ragged", op="attend", B=32, lo=512, hi=16384, hq=32, hkv=8, D=128, page=64, q="bf16",
             kv="bf16", window=0),
        # the largest batch: 64 long sequences in an 8-bit cache, groups of 16 query heads
        dict(name="attend-64-long-8bit", op="attend", B=64, lo=8192, hi=16384, hq=128, hkv=8, D=128, page=32, q="bf16",
             kv="e4m3", window=0),
        # output projection of one decode token, onto the residual
        dict(name="linear-decode-1", op="linear", T=1, N=4096, K=4096, x="bf16", y="bf16", bias=False, act="none",
             res=True),
        # quantised q/k/v projection of a batch of 32 with its bias
        dict(name="linear-decode-32-8bit", op="linear", T=32, N=6144, K=4096, x="e4m3", y="bf16", bias=True,
             act="none", res=False),
        # a prompt's dense projection with activation and residual
        dict(name="linear-prompt-8192", op="linear", T=8192, N=6144, K=4096, x="bf16", y="bf16", bias=True,
             act="gelu", res=True),
    ]


def _log(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["norm", "append", "attend", "linear"])
    if op == "norm":
        T, H = _log(rng, 1, 8192), _log(rng, 64, 8192)
        if rng.random() < 0.6:
            H = max(64, H // 64 * 64)
        T = max(1, min(T, NORM_ELEMS // H))
        x = rng.choice(["bf16", "f16", "f32"])
        return dict(op=op, T=T, H=H, x=x, res=rng.choice([x, "f32"]), y=rng.choice([x, "e4m3"]))
    if op == "append":
        hkv, g, D = rng.choice([1, 2, 4, 8]), rng.choice([1, 3, 4, 8]), rng.choice([64, 80, 96, 128, 256])
        T = min(_log(rng, 1, 8192), APPEND_ELEMS // ((g + 2) * hkv * D))
        x = rng.choice(["bf16", "f16"])
        return dict(op=op, T=T, hq=g * hkv, hkv=hkv, D=D, page=rng.choice([1, 7, 16, 32, 64, 128]), x=x,
                    kv=rng.choice([x, "e4m3"]), rot=rng.choice([D, D // 2]), interleaved=rng.random() < 0.3)
    if op == "attend":
        hkv, g, D = rng.choice([1, 2, 4, 8]), rng.choice([1, 3, 4, 7, 8, 16]), rng.choice([64, 96, 128, 192, 256])
        q = rng.choice(["bf16", "f16"])
        kv = rng.choice([q, "e4m3"])
        B = _log(rng, 1, 64)
        most = KV_BYTES // (2 * B * hkv * D * SIZE[kv])
        hi = _log(rng, 16, max(17, min(16384, most)))
        return dict(op=op, B=B, lo=rng.choice([0, 1, hi // 4, hi]), hi=hi, hq=g * hkv, hkv=hkv, D=D,
                    page=rng.choice([1, 7, 16, 32, 64, 128]), q=q, kv=kv,
                    window=rng.choice([0, 0, 0, 1 + hi // 3]))
    N, K = _log(rng, 64, 8192), max(64, _log(rng, 64, 8192) // 16 * 16)
    T = max(1, min(_log(rng, 1, 8192), MM_FLOPS // (2 * N * K)))
    return dict(op=op, T=T, N=N, K=K, x=rng.choice(["bf16", "f16", "e4m3"]), y=rng.choice(["bf16", "f16", "f32"]),
                bias=rng.random() < 0.5, act=rng.choice(["none", "relu", "gelu", "silu"]), res=rng.random() < 0.5)


def _lengths(case):
    """The batch's lengths: spread evenly from lo to hi, so that their sum is the case's own."""
    B, lo, hi = case["B"], case["lo"], case["hi"]
    return [hi if B == 1 else lo + (hi - lo) * i // (B - 1) for i in range(B)]


def _gen(seed):
    return torch.Generator(device="cuda").manual_seed(seed & 0x7FFFFFFF)


def _randn(g, *shape):
    return torch.randn(*shape, generator=g, device="cuda", dtype=torch.float32)


def _page_order(g, n):
    return torch.randperm(n, generator=g, device="cuda").to(torch.int32)


def _prepare_norm(c, g):
    T, H = c["T"], c["H"]
    s = dict(c, eps=EPS)
    s["xt"] = _randn(g, T, H).to(DT[c["x"]])
    # a residual stream has grown over the layers and has a few wide channels
    s["rt"] = (_randn(g, T, H) * 3.0 * torch.exp(0.5 * _randn(g, H))).to(DT[c["res"]])
    s["w"] = (1.0 + 0.2 * _randn(g, H)).to(DT[c["x"]])
    s["sum"] = torch.empty(T, H, dtype=DT[c["res"]], device="cuda")
    s["yt"] = torch.empty(T, H, dtype=DT[c["y"]], device="cuda")
    s["scale"] = torch.empty(T, dtype=torch.float32, device="cuda") if c["y"] == "e4m3" else None
    return s


def _rotation_table(positions, rot):
    inv = 10000.0 ** (-torch.arange(0, rot, 2, device="cuda", dtype=torch.float64) / rot)
    a = torch.arange(positions, device="cuda", dtype=torch.float64)[:, None] * inv
    return torch.cat([torch.cos(a), torch.sin(a)], 1).to(torch.float32)


def _prepare_append(c, g):
    T, hq, hkv, D, page = c["T"], c["hq"], c["hkv"], c["D"], c["page"]
    s = dict(c)
    # the three parts of a fused projection's rows
    qkv = _randn(g, T, hq + 2 * hkv, D).to(DT[c["x"]])
    s["qt"], s["kt"], s["vt"] = qkv[:, :hq], qkv[:, hq:hq + hkv], qkv[:, hq + hkv:]
    n_pages = -(-T // page) + 3
    order = _page_order(g, n_pages)
    t = torch.arange(T, device="cuda")
    s["slots"] = (order[t // page].to(torch.int64) * page + t % page).contiguous()
    s["pos"] = (t + 100).to(torch.int32)
    s["table"] = _rotation_table(T + 128, c["rot"])
    s["kc"] = _randn(g, n_pages, page, hkv, D).to(DT[c["kv"]])
    s["vc"] = _randn(g, n_pages, page, hkv, D).to(DT[c["kv"]])
    s["ks"] = s["vs"] = None
    if c["kv"] == "e4m3":
        s["ks"] = 0.01 + 0.01 * torch.rand(hkv, generator=g, device="cuda")
        s["vs"] = 0.01 + 0.01 * torch.rand(hkv, generator=g, device="cuda")
    s["qo"] = torch.empty(T, hq, D, dtype=DT[c["x"]], device="cuda")
    s["cache"] = _cache(s, hq, 1)
    return s


def _fill(cache, scale, g):
    v = _randn(g, *cache.shape)
    cache.copy_(v if scale is None else (v / scale[:, None]).clamp_(-E4M3_MAX, E4M3_MAX))


def _prepare_attend(c, g):
    B, hq, hkv, D, page = c["B"], c["hq"], c["hkv"], c["D"], c["page"]
    s = dict(c)
    lens = torch.tensor(_lengths(c), device="cuda")
    s["lens"] = lens[torch.randperm(B, generator=g, device="cuda")].to(torch.int32)
    per = max(1, -(-c["hi"] // page))
    need = (s["lens"].long() + page - 1) // page
    first = torch.cumsum(need, 0) - need
    n_pages = sum(-(-n // page) for n in _lengths(c)) + 2
    order = _page_order(g, n_pages)
    at = torch.arange(per, device="cuda")[None, :]
    # rows of pages past a sequence's end hold page 0, as an engine's table does
    s["pages"] = torch.where(at < need[:, None], order[(first[:, None] + at).clamp(max=n_pages - 1)],
                             torch.zeros((), dtype=torch.int32, device="cuda")).contiguous()
    s["qt"] = _randn(g, B, hq, D).to(DT[c["q"]])
    s["kc"] = torch.empty(n_pages, page, hkv, D, dtype=DT[c["kv"]], device="cuda")
    s["vc"] = torch.empty_like(s["kc"])
    s["ks"] = s["vs"] = None
    if c["kv"] == "e4m3":
        s["ks"] = 0.01 + 0.01 * torch.rand(hkv, generator=g, device="cuda")
        s["vs"] = 0.01 + 0.01 * torch.rand(hkv, generator=g, device="cuda")
    _fill(s["kc"], s["ks"], g)
    _fill(s["vc"], s["vs"], g)
    s["scale"] = 1.0 / math.sqrt(D)
    s["ot"] = torch.empty(B, hq, D, dtype=DT[c["q"]], device="cuda")
    s["lse"] = torch.empty(B, hq, dtype=torch.float32, device="cuda")
    s["cache"] = _cache(s, hq, B)
    return s


def _cache(s, hq, batch):
    """The cache handle that a user's program keeps."""
    if not own:
        return None
    import moe_decode_host_gb300 as m

    return m.KvCache(s["kc"], s["vc"], q_heads=hq, max_batch=batch, k_scale=s["ks"], v_scale=s["vs"])


def _prepare_linear(c, g):
    T, N, K = c["T"], c["N"], c["K"]
    s = dict(c)
    x, w = _randn(g, T, K), _randn(g, N, K) / math.sqrt(K)
    s["xs"] = s["ws"] = None
    if c["x"] == "e4m3":
        s["xs"] = x.abs().amax(1).clamp_(min=TINY) / E4M3_MAX
        s["ws"] = w.abs().amax(1).clamp_(min=TINY) / E4M3_MAX
        x, w = x / s["xs"][:, None], w / s["ws"][:, None]
    s["xt"], s["wt"] = x.to(DT[c["x"]]), w.to(DT[c["x"]])
    s["b"] = 0.1 * _randn(g, N) if c["bias"] else None
    s["rt"] = _randn(g, T, N).to(DT[c["y"]]) if c["res"] else None
    s["yt"] = torch.empty(T, N, dtype=DT[c["y"]], device="cuda")
    return s


def prepare(case, seed):
    return {"norm": _prepare_norm, "append": _prepare_append, "attend": _prepare_attend,
            "linear": _prepare_linear}[case["op"]](case, _gen(seed))


# ---- plain forms: 32 bits throughout, one rounding at the end -----------------


def _plain_norm(s):
    a = s["xt"].float() + s["rt"].float()
    y = a * torch.rsqrt((a * a).mean(1, keepdim=True) + s["eps"]) * s["w"].float()
    if s["scale"] is None:
        return [a.to(s["sum"].dtype), y.to(s["yt"].dtype)]
    scale = (y.abs().amax(1) / E4M3_MAX).clamp(min=TINY)
    return [a.to(s["sum"].dtype), (y / scale[:, None]).to(torch.float8_e4m3fn), scale]


def _rotated(x, table, rot, interleaved):
    cos, sin = table[:, None, : rot // 2], table[:, None, rot // 2:]
    y = x.clone()
    if interleaved:
        a, b = x[..., 0:rot:2], x[..., 1:rot:2]
        y[..., 0:rot:2], y[..., 1:rot:2] = a * cos - b * sin, a * sin + b * cos
    else:
        a, b = x[..., : rot // 2], x[..., rot // 2: rot]
        y[..., : rot // 2], y[..., rot // 2: rot] = a * cos - b * sin, a * sin + b * cos
    return y


def _plain_append(s):
    table = s["table"][s["pos"].long()]
    q = _rotated(s["qt"].float(), table, s["rot"], s["interleaved"])
    k = _rotated(s["kt"].float(), table, s["rot"], s["interleaved"])
    v = s["vt"].float()
    if s["ks"] is not None:
        k = (k / s["ks"][:, None]).clamp(-E4M3_MAX, E4M3_MAX)
        v = (v / s["vs"][:, None]).clamp(-E4M3_MAX, E4M3_MAX)
    page = s["page"]
    s["kc"][s["slots"] // page, s["slots"] % page] = k.to(s["kc"].dtype)
    s["vc"][s["slots"] // page, s["slots"] % page] = v.to(s["vc"].dtype)
    return [q.to(s["qo"].dtype), s["kc"], s["vc"]]


def _plain_attend(s):
    B, hq, hkv, D = s["B"], s["hq"], s["hkv"], s["D"]
    pages = s["pages"].long()
    k, v = s["kc"][pages].float(), s["vc"][pages].float()
    L = k.shape[1] * k.shape[2]
    k, v = k.view(B, L, hkv, D), v.view(B, L, hkv, D)
    if s["ks"] is not None:
        k, v = k.mul_(s["ks"][:, None]), v.mul_(s["vs"][:, None])
    q = s["qt"].float().view(B, hkv, hq // hkv, D)
    a = torch.matmul(q, k.permute(0, 2, 3, 1)) * s["scale"]
    at, n = torch.arange(L, device="cuda")[None, :], s["lens"].long()[:, None]
    seen = at < n
    if s["window"]:
        seen = seen & (at >= n - s["window"])
    a = a.masked_fill(~seen[:, None, None, :], -math.inf)
    top = a.amax(-1, keepdim=True)
    p = torch.exp(a - top.clamp(min=-3e38))
    total = p.sum(-1, keepdim=True)
    o = torch.matmul(p, v.permute(0, 2, 1, 3)) / total.clamp(min=1e-30)
    return [o.reshape(B, hq, D).to(s["ot"].dtype), (top + torch.log(total)).reshape(B, hq)]


def _activated(y, act):
    if act == "relu":
        return y.clamp(min=0)
    if act == "silu":
        return y / (1 + torch.exp(-y))
    if act == "gelu":
        return 0.5 * y * (1 + torch.erf(y / math.sqrt(2.0)))
    return y


def _plain_linear(s):
    y = torch.matmul(s["xt"].float(), s["wt"].float().t())
    if s["xs"] is not None:
        y = y * s["xs"][:, None] * s["ws"]
    if s["b"] is not None:
        y = y + s["b"]
    y = _activated(y, s["act"])
    if s["rt"] is not None:
        y = y + s["rt"].float()
    return y.to(s["yt"].dtype)


# ---- the library's entry points ----------------------------------------------


def _own(s):
    import moe_decode_host_gb300 as m

    op = s["op"]
    if op == "norm":
        m.moe_add_rms_norm(s["xt"], s["w"], s["yt"], residual=s["rt"], sum_out=s["sum"], scale=s["scale"],
                           eps=s["eps"])
        return [s["sum"], s["yt"]] + ([] if s["scale"] is None else [s["scale"]])
    if op == "append":
        m.moe_kv_append(s["cache"], s["qt"], s["kt"], s["vt"], s["pos"], s["slots"], s["table"], s["qo"],
                        interleaved=s["interleaved"])
        return [s["qo"], s["kc"], s["vc"]]
    if op == "attend":
        m.moe_kv_attend(s["cache"], s["qt"], s["pages"], s["lens"], s["ot"], scale=s["scale"], window=s["window"],
                        lse=s["lse"])
        return [s["ot"], s["lse"]]
    m.moe_linear(s["xt"], s["wt"], s["yt"], bias=s["b"], act=s["act"], residual=s["rt"], x_scale=s["xs"],
                 w_scale=s["ws"])
    return s["yt"]


def run(state):
    if own:
        return _own(state)
    return {"norm": _plain_norm, "append": _plain_append, "attend": _plain_attend,
            "linear": _plain_linear}[state["op"]](state)


def work(case):
    op = case["op"]
    if op == "norm":
        T, H = case["T"], case["H"]
        b = T * H * (SIZE[case["x"]] + 2 * SIZE[case["res"]] + SIZE[case["y"]]) + H * SIZE[case["x"]]
        return {"bytes": b + (4 * T if case["y"] == "e4m3" else 0), "flops": 5 * T * H}
    if op == "append":
        T, hq, hkv, D = case["T"], case["hq"], case["hkv"], case["D"]
        b = T * D * (2 * hq * SIZE[case["x"]] + 2 * hkv * (SIZE[case["x"]] + SIZE[case["kv"]]))
        return {"bytes": b + T * (12 + 4 * case["rot"]), "flops": 3 * T * (hq + hkv) * case["rot"]}
    if op == "attend":
        n = sum(min(v, case["window"]) if case["window"] else v for v in _lengths(case))
        B, hq, hkv, D = case["B"], case["hq"], case["hkv"], case["D"]
        b = 2 * n * hkv * D * SIZE[case["kv"]] + B * hq * (2 * D * SIZE[case["q"]] + 4)
        return {"bytes": b + 4 * n // case["page"] + 4 * B, "flops": 4 * n * hq * D}
    T, N, K = case["T"], case["N"], case["K"]
    b = (T + N) * K * SIZE[case["x"]] + T * N * SIZE[case["y"]] * (2 if case["res"] else 1)
    b += 4 * N if case["bias"] else 0
    b += 4 * (T + N) if case["x"] == "e4m3" else 0
    return {"bytes": b, "flops": 2 * T * N * K}


# ---- definitions in 64 bits ----------------------------------------------------


def _exact_norm(s):
    h = s["xt"].double() + s["rt"].double()
    ms = torch.einsum("th,th->t", h, h) / s["H"] + s["eps"]
    y = h / torch.sqrt(ms)[:, None] * s["w"].double()[None, :]
    if s["scale"] is None:
        return [h, y]
    scale = torch.maximum(y.abs().max(1).values / 448, torch.tensor(TINY, dtype=torch.float64, device="cuda"))
    return [h, y / scale[:, None], scale]


def _exact_turn(x, cs, rot, interleaved):
    """Each pair as a complex number, turned by its angle."""
    turn = torch.complex(cs[:, : rot // 2], cs[:, rot // 2:])[:, None, :]
    head, tail = x[..., :rot], x[..., rot:]
    if interleaved:
        z = torch.view_as_complex(head.reshape(*head.shape[:-1], rot // 2, 2).contiguous()) * turn
        head = torch.view_as_real(z).reshape(head.shape)
    else:
        z = torch.complex(head[..., : rot // 2].contiguous(), head[..., rot // 2:].contiguous()) * turn
        head = torch.cat([z.real, z.imag], -1)
    return torch.cat([head, tail], -1)


def _exact_append(s):
    cs = s["table"].double()[s["pos"].long()]
    q = _exact_turn(s["qt"].double(), cs, s["rot"], s["interleaved"])
    k = _exact_turn(s["kt"].double(), cs, s["rot"], s["interleaved"])
    v = s["vt"].double()
    if s["ks"] is not None:
        k = torch.clamp(k / s["ks"].double()[None, :, None], -448, 448)
        v = torch.clamp(v / s["vs"].double()[None, :, None], -448, 448)
    shape, width = s["kc"].shape, s["hkv"] * s["D"]
    kc, vc = s["kc"].double().reshape(-1, width), s["vc"].double().reshape(-1, width)
    kc.index_copy_(0, s["slots"], k.reshape(-1, width))
    vc.index_copy_(0, s["slots"], v.reshape(-1, width))
    return [q, kc.view(shape), vc.view(shape)]


def _exact_sequence(s, b, n):
    """One sequence over its own tokens alone."""
    hq, hkv, D, page = s["hq"], s["hkv"], s["D"], s["page"]
    first = max(0, n - s["window"]) if s["window"] else 0
    if n <= first:
        return (torch.zeros(hq, D, dtype=torch.float64, device="cuda"),
                torch.full((hq,), -math.inf, dtype=torch.float64, device="cuda"))
    t = torch.arange(first, n, device="cuda")
    where = s["pages"][b].long()[t // page] * page + t % page
    k, v = s["kc"].reshape(-1, hkv, D)[where].double(), s["vc"].reshape(-1, hkv, D)[where].double()
    if s["ks"] is not None:
        k, v = k * s["ks"].double()[:, None], v * s["vs"].double()[:, None]
    q = s["qt"][b].double().reshape(hkv, hq // hkv, D)
    a = torch.einsum("hgd,thd->hgt", q, k) * s["scale"]
    z = torch.logsumexp(a, -1)
    return torch.einsum("hgt,thd->hgd", torch.exp(a - z[..., None]), v).reshape(hq, D), z.reshape(hq)


def _exact_attend(s):
    each = [_exact_sequence(s, b, n) for b, n in enumerate(s["lens"].tolist())]
    return [torch.stack([o for o, _ in each]), torch.stack([z for _, z in each])]


def _exact_linear(s):
    x, w = s["xt"].double(), s["wt"].double()
    if s["xs"] is not None:
        x, w = x * s["xs"].double()[:, None], w * s["ws"].double()[:, None]
    y = torch.einsum("tk,nk->tn", x, w)
    if s["b"] is not None:
        y = y + s["b"].double()
    if s["act"] == "relu":
        y = torch.relu(y)
    elif s["act"] == "silu":
        y = y * torch.sigmoid(y)
    elif s["act"] == "gelu":
        y = y * torch.special.ndtr(y)
    return y if s["rt"] is None else y + s["rt"].double()


def exact(case, seed):
    s = prepare(case, seed)
    return {"norm": _exact_norm, "append": _exact_append, "attend": _exact_attend,
            "linear": _exact_linear}[case["op"]](s)
