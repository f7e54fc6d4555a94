"""What the serving operators around a growing KV cache are measured on.

Four operators of one step of decoding with drafted tokens: rotary positions
(`rope`), the cache written in 16 or 8 bits and read back (`append`, `read`),
and attention of a tree of drafted tokens over that cache (`attn`).  With
`own` false, run() computes them in plain torch operations; with `own` true
it makes the calls a user makes of token_level_dynamic_b200.
"""
import math

import numpy as np
import torch

own = False

HD = 128                 # head dimension of the cache and the attention
BLOCK = 32               # cache elements that share one scale
KINDS = ("bf16", "e4m3", "i8")


def listed():
    return [
        # one decoding step of a small batch: q and k heads of 8 sequences' tokens, where latency counts
        dict(name="rope decode step", op="rope", tokens=8, heads=40, head_dim=128, rot_dim=128,
             layout="half", dtype="bf16", scaling="none", far=4096),
        # a prefill's q and k heads with frequencies scaled for a long context, at far positions
        dict(name="rope prefill scaled", op="rope", tokens=8192, heads=40, head_dim=128, rot_dim=128,
             layout="half", dtype="bf16", scaling="ramp", far=1000000),
        # interleaved pairs over part of the head, in 32 bits, odd token count
        dict(name="rope partial interleaved", op="rope", tokens=2311, heads=24, head_dim=96, rot_dim=36,
             layout="interleaved", dtype="f32", scaling="linear", far=60000),
        # one token of each of 16 sequences into an 8-bit cache, keys rotated on the way
        dict(name="append decode e4m3", op="append", n_seq=16, seq_len=1, n_kv=8, cap=2112, kind="e4m3",
             rope="half", ragged=True),
        # a prefill's keys and values into an 8-bit cache
        dict(name="append prefill i8", op="append", n_seq=4, seq_len=2048, n_kv=8, cap=2112, kind="i8",
             rope="none", ragged=False),
        # ragged sequences of an 8-bit cache back in bf16, as a caller moves them elsewhere
        dict(name="read ragged e4m3", op="read", n_seq=7, seq_len=6001, n_kv=8, cap=6144, kind="e4m3",
             ragged=True),
        # one token of one sequence over a bf16 cache: the smallest step
        dict(name="attn one token bf16", op="attn", n_seq=1, draft=1, n_kv=8, rep=4, length=2048,
             kind="bf16", tree=False, keep=1.0, ragged=False),
        # a batch that verifies small trees, a third of the head groups kept
        dict(name="attn small trees e4m3", op="attn", n_seq=16, draft=8, n_kv=8, rep=4, length=2048,
             kind="e4m3", tree=True, keep=0.34, ragged=False),
        # ragged batch, odd tree, three query heads to a key head
        dict(name="attn ragged i8", op="attn", n_seq=29, draft=5, n_kv=8, rep=3, length=8191,
             kind="i8", tree=True, keep=1.0, ragged=True),
        # long context, a chain of drafted tokens
        dict(name="attn long context e4m3", op="attn", n_seq=1, draft=16, n_kv=8, rep=4, length=131056,
             kind="e4m3", tree=False, keep=1.0, ragged=False),
        # wide trees over bf16 caches: the tensor cores count
        dict(name="attn wide trees bf16", op="attn", n_seq=8, draft=61, n_kv=8, rep=4, length=8000,
             kind="bf16", tree=True, keep=0.5, ragged=True),
        # the largest: wide trees over long 8-bit caches
        dict(name="attn wide trees i8", op="attn", n_seq=4, draft=64, n_kv=8, rep=4, length=32000,
             kind="i8", tree=True, keep=1.0, ragged=False),
    ]


def _log(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(("rope", "append", "read", "attn", "attn", "attn"))
    if op == "rope":
        head_dim = rng.choice((64, 80, 96, 128, 128, 256))
        rot = rng.choice((head_dim, head_dim, head_dim // 2, 2 * rng.randint(1, head_dim // 2)))
        heads = rng.randint(1, 48)
        return dict(op=op, tokens=_log(rng, 1, max(1, 8192 * 40 * 128 // (heads * head_dim * 2))),
                    heads=heads, head_dim=head_dim, rot_dim=rot,
                    layout=rng.choice(("half", "interleaved")), dtype=rng.choice(("bf16", "bf16", "f32")),
                    scaling=rng.choice(("none", "linear", "ramp")), far=_log(rng, 1, 1 << 21))
    if op in ("append", "read"):
        n_seq, n_kv = rng.randint(1, 32), rng.randint(1, 16)
        seq_len = _log(rng, 1, max(1, 65536 // (n_seq * n_kv)))
        c = dict(op=op, n_seq=n_seq, seq_len=seq_len, n_kv=n_kv, cap=seq_len + rng.randint(0, 97),
                 kind=rng.choice(KINDS), ragged=rng.random() < 0.5)
        if op == "append":
            c["rope"] = rng.choice(("none", "half", "interleaved"))
        return c
    rep, n_kv = rng.choice((1, 2, 3, 4, 4, 8)), rng.choice((1, 2, 4, 8, 8, 16))
    n_seq, draft = _log(rng, 1, 32), _log(rng, 1, 64)
    # rows x positions and cache bytes both stay within those of the largest listed case
    most = min(131000, (4 * 64 * 32 * 32000) // (n_seq * draft * rep * n_kv),
               (4 * 8 * 32000) // (n_seq * n_kv))
    return dict(op=op, n_seq=n_seq, draft=draft, n_kv=n_kv, rep=rep, length=_log(rng, 1, max(1, most)),
                kind=rng.choice(KINDS), tree=rng.random() < 0.6, keep=rng.choice((1.0, 1.0, 0.5, 0.34)),
                ragged=rng.random() < 0.5)


# ------------------------------------------------------------------ inputs

def _lens(case):
    """(tokens already in the cache, drafted or new tokens) of each sequence, fixed by the case."""
    s = np.arange(case["n_seq"])
    if case["op"] == "attn":
        new, old = np.full(len(s), case["draft"]), np.full(len(s), case["length"])
    else:
        new = np.full(len(s), case["seq_len"])
        old = np.full(len(s), case["cap"] - case["seq_len"] if case["op"] == "append" else 0)
    if case["ragged"]:
        new = np.maximum(new - s % 3, 0) if case["op"] != "read" else new * (len(s) - s) // len(s)
        old = old * (len(s) - s) // len(s)
    return old.astype(np.int32), new.astype(np.int32)


def _trees(rng, n_seq, n):
    """Ancestor-or-self matrices [n_seq][n][n] of random trees: token i's parent is one of the four before it, or the context."""
    a = np.zeros((n_seq, n, n), dtype=bool)
    at = np.arange(n_seq)
    for i in range(n):
        parent = rng.integers(max(i - 4, -1), i, n_seq) if i else np.full(n_seq, -1)
        a[:, i] = np.where(parent[:, None] >= 0, a[at, np.maximum(parent, 0)], False)
        a[:, i, i] = True
    return a


def _words(bits):
    """Truth values [...][n] as 32-bit words [...][ceil(n / 32)], bit i of word w for column 32 w + i."""
    n = bits.shape[-1]
    pad = np.zeros(bits.shape[:-1] + (-(-n // 32) * 32,), dtype=np.uint8)
    pad[..., :n] = bits
    return np.packbits(pad, axis=-1, bitorder="little").view(np.uint32).view(np.int32)


def _rope_of(case):
    """Rotary parameters: base, frequency scaling and its numbers, amplitude."""
    kind = case.get("scaling", "none")
    return dict(theta=500000.0, factor=1.0 if kind == "none" else 8.0, low=1.0 if kind == "ramp" else 0.0,
                high=4.0 if kind == "ramp" else 0.0, original=8192 if kind == "ramp" else 0,
                amplitude=1.0 + 0.1 * math.log(8.0) if kind == "ramp" else 1.0)


def _like_keys(shape, g, device):
    """Values with a few channels several times the others, as keys have them."""
    x = torch.randn(shape, generator=g, device=device)
    return x * torch.where(torch.rand(shape[-1], generator=g, device=device) < 0.04, 6.0, 1.0)


def prepare(case, seed):
    dev = "cuda"
    g = torch.Generator(device=dev).manual_seed(seed)
    rng = np.random.default_rng(seed)
    up = lambda a: torch.from_numpy(np.ascontiguousarray(a)).to(dev)  # noqa: E731
    st = dict(case)
    if case["op"] == "rope":
        dt = torch.bfloat16 if case["dtype"] == "bf16" else torch.float32
        st["x"] = torch.randn((case["tokens"], case["heads"], case["head_dim"]), generator=g, device=dev).to(dt)
        st["positions"] = up(rng.integers(0, case["far"], case["tokens"]).astype(np.int32))
        st["rope_cfg"] = _rope_of(case)
        return st
    n_seq, n_kv = case["n_seq"], case["n_kv"]
    old, new = _lens(case)
    n = case["draft"] if case["op"] == "attn" else case["seq_len"]
    cap = int((old + new).max()) + 3 if case["op"] == "attn" else case["cap"]
    st["cap"], st["tokens_per_seq"] = cap, n
    st["old"], st["new"] = up(old), up(new)
    # the cache as earlier steps left it (for append: zeros)
    shape = (n_seq, n_kv, cap, HD)
    if case["op"] == "append":
        k = v = torch.zeros(shape, device=dev)
    else:
        k, v = _like_keys(shape, g, dev), torch.randn(shape, generator=g, device=dev)
    st["cache"] = {}
    for name, x in (("k", k), ("v", v)):
        x = x.to(torch.bfloat16)
        if case["kind"] == "bf16":
            st["cache"][name] = x.clone()
        else:
            st["cache"][name], st["cache"][name + "_scale"] = _quantised(x.float(), case["kind"])
        del x
    del k, v
    if case["op"] == "append":
        t = n_seq * n
        st["k"] = _like_keys((t, n_kv, HD), g, dev).to(torch.bfloat16)
        st["v"] = torch.randn((t, n_kv, HD), generator=g, device=dev).to(torch.bfloat16)
        st["rope_cfg"] = _rope_of({"scaling": "ramp"})
    if case["op"] in ("append", "read"):   # rows past a sequence's tokens stay as they are
        st["k_out"] = torch.zeros((n_seq * n, n_kv, HD), dtype=torch.bfloat16, device=dev)
        st["v_out"] = torch.zeros_like(st["k_out"])
        return st
    t, n_q = n_seq * n, n_kv * case["rep"]
    st["q"] = (2.0 * torch.randn((t, n_q, HD), generator=g, device=dev)).to(torch.bfloat16)
    st["tree"] = up(_words(_trees(rng, n_seq, n)).reshape(t, -1)) if case["tree"] else None
    st["heads"] = up(_words(rng.random((t, n_kv)) < case["keep"])) if case["keep"] < 1.0 else None
    st["out"] = torch.zeros((t, n_q, HD), dtype=torch.bfloat16, device=dev)
    return st


# -------------------------------------------------------------- plain forms

def _quantised(x, kind):
    """Codes of x (fp32 [..., HD]) and one power-of-two scale per BLOCK elements, held as exponent + 127:
    the smallest that the block's largest value does not overflow; 255 and zero codes where a value is not finite."""
    most = 448.0 if kind == "e4m3" else 127.0
    b = x.unflatten(-1, (-1, BLOCK))
    top = b.abs().amax(-1)
    e = torch.frexp(top)[1] - (9 if kind == "e4m3" else 7)
    e = torch.clamp(e + (torch.ldexp(top, -e) > most).int(), min=-124)
    e = torch.where(top == 0, torch.full_like(e, -127), e)
    y = torch.ldexp(b, -e[..., None])
    bad = ~torch.isfinite(top)
    y = torch.where(bad[..., None] | (top == 0)[..., None], torch.zeros_like(y), y).flatten(-2)
    codes = y.to(torch.float8_e4m3fn) if kind == "e4m3" else torch.round(y).to(torch.int8)
    return codes, torch.where(bad, torch.full_like(e, 255), e + 127).to(torch.uint8)


def _values(cache, name):
    """The numbers a cache stands for, in fp32."""
    x = cache[name].float()
    if name + "_scale" not in cache:
        return x
    s = cache[name + "_scale"].int()
    f = torch.where(s == 255, torch.full_like(s, 0, dtype=torch.float32) * float("nan"),
                    torch.ldexp(torch.ones_like(s, dtype=torch.float32), s - 127))
    return (x.unflatten(-1, (-1, BLOCK)) * f[..., None]).flatten(-2)


def _frequencies(cfg, rot_dim, device):
    """Radians per position of each pair, in 64 bits."""
    i = torch.arange(rot_dim // 2, dtype=torch.float64, device=device)
    f = torch.exp(-math.log(cfg["theta"]) * 2.0 * i / rot_dim)
    if cfg["factor"] == 1.0:
        return f
    if cfg["original"] == 0:
        return f / cfg["factor"]
    turns = cfg["original"] * f / (2.0 * math.pi)
    keep = torch.clamp((turns - cfg["low"]) / (cfg["high"] - cfg["low"]), 0.0, 1.0)
    return f * (keep + (1.0 - keep) / cfg["factor"])


def _rotated(x, positions, cfg, rot_dim, layout):
    """x (fp32 [T][n][head_dim]) with its first rot_dim elements rotated by the tokens' positions."""
    ang = positions.double()[:, None] * _frequencies(cfg, rot_dim, x.device)
    cs = (ang.cos() * cfg["amplitude"]).float()[:, None]
    sn = (ang.sin() * cfg["amplitude"]).float()[:, None]
    r, rest = x[..., :rot_dim], x[..., rot_dim:]
    if layout == "half":
        a, b = r[..., : rot_dim // 2], r[..., rot_dim // 2:]
        return torch.cat((a * cs - b * sn, b * cs + a * sn, rest), -1)
    a, b = r[..., 0::2], r[..., 1::2]
    return torch.cat((torch.stack((a * cs - b * sn, b * cs + a * sn), -1).flatten(-2), rest), -1)


def _rows_of(st):
    """Sequence and cache position of every token, and which tokens there are."""
    n = st["tokens_per_seq"]
    t = torch.arange(st["n_seq"] * n, device=st["old"].device)
    s, i = t // n, t % n
    start = torch.zeros_like(st["old"]) if st["op"] == "read" else st["old"]
    return s, start[s] + i, i < st["new"][s]


def _plain_read(st):
    s, pos, there = _rows_of(st)
    s, pos = s[there], pos[there].long()
    for name, out in (("k", st["k_out"]), ("v", st["v_out"])):
        rows = {x: st["cache"][x][s, :, pos] for x in st["cache"] if x.startswith(name)}
        out[there] = _values(rows, name).to(torch.bfloat16)
    return st["k_out"], st["v_out"]


def _plain_append(st):
    s, pos, there = _rows_of(st)
    k, v = st["k"].float(), st["v"].float()
    if st["rope"] != "none":
        k = _rotated(k, pos, st["rope_cfg"], HD, st["rope"])
    s, pos = s[there], pos[there].long()
    for name, x in (("k", k[there]), ("v", v[there])):
        if st["kind"] == "bf16":
            st["cache"][name][s, :, pos] = x.to(torch.bfloat16)
        else:
            codes, scale = _quantised(x, st["kind"])
            st["cache"][name].view(torch.uint8)[s, :, pos] = codes.view(torch.uint8)
            st["cache"][name + "_scale"][s, :, pos] = scale
    return _plain_read(st)


def _bits(words, n):
    i = torch.arange(n, device=words.device)
    return ((words[:, i // 32] >> (i % 32).int()) & 1).bool()


def _plain_attn(st):
    n_seq, n, n_kv, rep, cap = st["n_seq"], st["draft"], st["n_kv"], st["rep"], st["cap"]
    dev = st["q"].device
    k, v = _values(st["cache"], "k"), _values(st["cache"], "v")
    q = st["q"].float().view(n_seq, n, n_kv, rep, HD).permute(0, 2, 1, 3, 4).reshape(n_seq, n_kv, n * rep, HD)
    j = torch.arange(cap, device=dev)[None] - st["old"][:, None]              # place among the drafted tokens
    i = torch.arange(n, device=dev)
    tree = (i[None, :] <= i[:, None]).expand(n_seq, n, n) if st["tree"] is None else _bits(st["tree"], n).view(n_seq, n, n)
    seen = tree.gather(2, j.clamp(0, n - 1)[:, None].expand(n_seq, n, cap))
    seen = torch.where((j < 0)[:, None], True, seen & (j < st["new"][:, None])[:, None])
    s = (q @ k.transpose(-1, -2)) * (1.0 / math.sqrt(HD))
    s.view(n_seq, n_kv, n, rep, cap).masked_fill_(~seen[:, None, :, None], -math.inf)
    top = s.amax(-1, keepdim=True)
    p = torch.exp(s - torch.where(torch.isfinite(top), top, torch.zeros_like(top)))
    del s
    total = p.sum(-1, keepdim=True)
    o = (p @ v) / torch.where(total == 0, torch.ones_like(total), total)
    o = o.view(n_seq, n_kv, n, rep, HD).permute(0, 2, 1, 3, 4).reshape(n_seq * n, n_kv, rep, HD)
    if st["heads"] is not None:
        o = torch.where(_bits(st["heads"], n_kv)[:, :, None, None], o, torch.zeros_like(o))
    there = (i[None] < st["new"][:, None]).reshape(-1)
    st["out"][there] = o.reshape(n_seq * n, n_kv * rep, HD)[there].to(torch.bfloat16)
    return st["out"]


# ---------------------------------------------------------- the framework's

def _own(st):
    import token_level_dynamic_b200 as w

    layout = {"half": w.WIDE_ROPE_HALF, "interleaved": w.WIDE_ROPE_INTERLEAVED}
    if st["op"] == "rope" or st.get("rope", "none") != "none":
        c = st["rope_cfg"]
        cfg = w.wide_rope_config(st.get("rot_dim", HD), c["theta"], layout[st.get("layout", st.get("rope"))],
                                 factor=c["factor"], low_freq=c["low"], high_freq=c["high"],
                                 original_len=c["original"], amplitude=c["amplitude"])
    if st["op"] == "rope":
        return w.wide_rope(st["x"], st["positions"], cfg)
    if st["op"] == "append":
        w.wide_kv_append(st["k"], st["v"], st["cache"], st["old"], count=st["new"],
                         rope=cfg if st["rope"] != "none" else None)
        return w.wide_kv_read(st["cache"], st["old"], st["seq_len"], count=st["new"], k=st["k_out"], v=st["v_out"])
    if st["op"] == "read":
        return w.wide_kv_read(st["cache"], None, st["seq_len"], count=st["new"], k=st["k_out"], v=st["v_out"])
    return w.wide_attn_tree(st["q"], st["cache"], st["old"], tree_mask=st["tree"], head_mask=st["heads"],
                            draft_len=st["new"], out=st["out"])


def run(state):
    if own:
        return _own(state)
    if state["op"] == "rope":
        return _rotated(state["x"].float(), state["positions"], state["rope_cfg"], state["rot_dim"],
                        state["layout"]).to(state["x"].dtype)
    return {"append": _plain_append, "read": _plain_read, "attn": _plain_attn}[state["op"]](state)


# -------------------------------------------------------------------- work

def work(case):
    if case["op"] == "rope":
        n = case["tokens"] * case["heads"] * case["head_dim"]
        return {"bytes": 2 * n * (2 if case["dtype"] == "bf16" else 4) + 4 * case["tokens"],
                "flops": 3 * case["tokens"] * case["heads"] * case["rot_dim"]}
    row = HD * 2 if case["kind"] == "bf16" else HD + HD // BLOCK      # bytes of one row of the cache
    old, new = _lens(case)
    if case["op"] in ("append", "read"):
        rows = 2 * int(new.sum()) * case["n_kv"]
        # read: the cache's rows in, bf16 rows out; append: bf16 rows in, the cache's rows out, then that read
        return {"bytes": rows * (row + HD * 2) * (2 if case["op"] == "append" else 1) + 8 * case["n_seq"],
                "flops": rows * HD}
    live = 1.0 - (1.0 - case["keep"]) ** new.astype(np.float64)       # pairs of sequence and group with a token
    kept = case["keep"] * new.astype(np.float64)                      # tokens of a group
    n_kv, rep = case["n_kv"], case["rep"]
    q_out = float(new.sum()) * n_kv * rep * HD * 2 * (1.0 + case["keep"])
    return {"bytes": float(((old + new) * live).sum()) * n_kv * 2 * row + q_out,
            "flops": float(((old + new) * kept).sum()) * n_kv * rep * HD * 4}


# ------------------------------------------------------- definition, 64 bits

def _exact_pairs(x, positions, cfg, rot_dim, layout):
    """Rotation as multiplication of complex numbers."""
    i = torch.arange(rot_dim // 2, dtype=torch.float64, device=x.device)
    f = cfg["theta"] ** (-(2.0 / rot_dim) * i)
    if cfg["original"]:
        r = cfg["original"] / (2.0 * math.pi / f)
        mix = ((r - cfg["low"]) / (cfg["high"] - cfg["low"])).clamp(0.0, 1.0)
        f = (1.0 - mix) * f / cfg["factor"] + mix * f
    else:
        f = f / cfg["factor"]
    w = torch.polar(torch.full((), cfg["amplitude"], dtype=torch.float64, device=x.device).expand(len(positions), len(f)).contiguous(),
                    positions.double()[:, None] * f[None])[:, None]
    out = x.double().clone()
    if layout == "half":
        z = torch.complex(out[..., : rot_dim // 2].contiguous(), out[..., rot_dim // 2: rot_dim].contiguous()) * w
        out[..., : rot_dim // 2], out[..., rot_dim // 2: rot_dim] = z.real, z.imag
    else:
        z = torch.complex(out[..., 0:rot_dim:2].contiguous(), out[..., 1:rot_dim:2].contiguous()) * w
        out[..., 0:rot_dim:2], out[..., 1:rot_dim:2] = z.real, z.imag
    return out


def _exact_rounded(x, kind):
    """x (64 bits) as an 8-bit block holds it: a power-of-two scale, then the nearest representable multiple, ties to even."""
    if kind == "bf16":
        step = torch.exp2((torch.frexp(x.abs().clamp(min=2.0 ** -126))[1] - 8).double())
        return torch.round(x / step) * step
    b = x.reshape(*x.shape[:-1], HD // BLOCK, BLOCK)
    top = b.abs().amax(-1, keepdim=True)
    m, e = torch.frexp(top.clamp(min=2.0 ** -120) / (448.0 if kind == "e4m3" else 127.0))
    s = torch.exp2((e - (m == 0.5).to(e.dtype)).double())      # the smallest power of two that is not below the ratio
    y = b / s
    if kind == "e4m3":
        step = torch.exp2((torch.frexp(y.abs().clamp(min=2.0 ** -6))[1] - 4).double())
        y = torch.round(y / step) * step
    else:
        y = torch.round(y)
    return (y * s).reshape(x.shape)


def _exact_cache(cache, name):
    x = cache[name].double()
    if name + "_scale" in cache:
        x = x * torch.exp2(cache[name + "_scale"].double() - 127.0).repeat_interleave(BLOCK, -1)
    return x


def exact(case, seed):
    st = prepare(case, seed)
    if case["op"] == "rope":
        return _exact_pairs(st["x"], st["positions"], st["rope_cfg"], case["rot_dim"], case["layout"])
    old, new = _lens(case)
    n, n_kv = st["tokens_per_seq"], case["n_kv"]
    if case["op"] in ("append", "read"):
        outs = []
        if case["op"] == "append":
            pos = torch.from_numpy((old[:, None] + np.arange(n)[None]).reshape(-1)).to("cuda")
            k, v = st["k"].double(), st["v"].double()
            if case["rope"] != "none":
                k = _exact_pairs(k, pos, st["rope_cfg"], HD, case["rope"])
            outs = [_exact_rounded(k, case["kind"]), _exact_rounded(v, case["kind"])]
        else:
            outs = [_exact_cache(st["cache"], name)[:, :, :n].transpose(1, 2).reshape(-1, n_kv, HD) for name in "kv"]
        for o in outs:
            for s in range(case["n_seq"]):
                o[s * n + int(new[s]): (s + 1) * n] = 0.0
        return tuple(outs)
    out = torch.zeros(st["out"].shape, dtype=torch.float64, device="cuda")
    k, v = (_exact_cache(st["cache"], name) for name in "kv")
    tree = None if st["tree"] is None else st["tree"].cpu().numpy().view(np.uint32)
    heads = None if st["heads"] is None else st["heads"].cpu().numpy().view(np.uint32)
    for s in range(case["n_seq"]):
        have, m = int(old[s]), int(new[s])
        if have + m == 0 or m == 0:
            continue
        sees = torch.ones((m, have + m), dtype=torch.bool)
        for t in range(m):
            for j in range(m):
                sees[t, have + j] = bool(j <= t if tree is None else (int(tree[s * n + t, j // 32]) >> (j % 32)) & 1)
        sees = sees.to("cuda")
        for h in range(n_kv):
            q = st["q"][s * n: s * n + m, h * case["rep"]: (h + 1) * case["rep"]].double()
            x = torch.einsum("trd,pd->trp", q, k[s, h, : have + m]) / math.sqrt(HD)
            x = x.masked_fill(~sees[:, None], -math.inf)
            o = torch.einsum("trp,pd->trd", torch.softmax(x, -1).nan_to_num(0.0), v[s, h, : have + m])
            if heads is not None:
                on = torch.from_numpy(((heads[s * n: s * n + m, h // 32] >> (h % 32)) & 1).astype(bool)).to("cuda")
                o = torch.where(on[:, None, None], o, torch.zeros_like(o))
            out[s * n: s * n + m, h * case["rep"]: (h + 1) * case["rep"]] = o
    return out
