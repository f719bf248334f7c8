"""The operators around the attention calls, as their users call them: what is timed, and what it is compared with.

Between a model's projections and the attention calls of this library lie the rotation of queries and keys by
their positions (with or without a norm of each head before it), the writing of keys and values into an 8-bit
paged cache, the reading back of that cache, and the attention of a chunk of new tokens over it.  Each case below
is one such call; `run` makes it once, in its plain form (elementary torch operations, 32 bits, rounded once) or,
where `own` is set, through the library.

Kinds of case:

* ``rope``           rotation of q and k (``transpose``: its gradient);
* ``norm_rope``      RMS norm of every head of q and k, then the rotation;
* ``norm_rope_bwd``  the gradients of that, of the norm's two weights too;
* ``kv_write``       quantise a chunk's keys and values into the pages of each sequence;
* ``kv_read``        the last tokens of each sequence out of the pages, as dense bf16;
* ``prefill``        attention of each sequence's chunk over its 8-bit pages.
"""
import math

import numpy as np
import torch

own = False

DEV = "cuda"
PAGE = 16
QMAX = {"e4m3": 448.0, "int8": 127.0}
CODES = {"e4m3": torch.float8_e4m3fn, "int8": torch.int8}
DTYPES = {"bf16": torch.bfloat16, "f32": torch.float32}
TINY = 2.0 ** -126  # the smallest page scale: that of a slice of zeros


# ------------------------------------------------------------------ the cases

def listed():
    rot = dict(hq=32, hkv=8, d=128, rot=128, interleaved=False, dtype="bf16", base=10000.0, factor=1.0, far=8192)
    cache = dict(hq=32, hkv=8, d=128, lengths=7)
    return [
        # One decode step of 64 sequences: one token each, at far positions of a context stretched fourfold.
        dict(rot, name="rope_decode_64", kind="rope", layout="tokens", b=1, n=64, factor=4.0, far=131072, transpose=False),
        # The gradient of a partial, interleaved rotation in the fp32 path, an odd length.
        dict(rot, name="rope_grad_f32_odd", kind="rope", layout="heads", b=2, n=2047, hq=16, hkv=16, d=64, rot=32,
             interleaved=True, dtype="f32", transpose=True),
        # One decode step with normed heads.
        dict(rot, name="norm_rope_decode_64", kind="norm_rope", layout="tokens", b=1, n=64),
        # A whole batch of prompts: the grouped-query prefill workload's q and k.
        dict(rot, name="norm_rope_prompt", kind="norm_rope", layout="heads", b=4, n=4096),
        # The same batch in training: gradients of q, k and both weights.
        dict(rot, name="norm_rope_bwd_train", kind="norm_rope_bwd", layout="heads", b=4, n=4096),
        # A small fp32 gradient, a quarter of each head rotated, an odd number of tokens.
        dict(rot, name="norm_rope_bwd_f32_odd", kind="norm_rope_bwd", layout="tokens", b=1, n=1021, hq=12, hkv=4, d=64,
             rot=16, interleaved=True, dtype="f32"),
        # One decode step writes 64 tokens into 64 half-filled pages: latency.
        dict(cache, name="kv_write_decode_64", kind="kv_write", s=64, qlo=1, qhi=1, clo=0, chi=8191, fmt="e4m3"),
        # A step of chunked prefill writes 512 tokens to each of 16 sequences, at unaligned places.
        dict(cache, name="kv_write_chunks", kind="kv_write", s=16, qlo=512, qhi=512, clo=0, chi=7680, fmt="int8"),
        # Two short prefixes are read back for a step that needs them dense.
        dict(cache, name="kv_read_short", kind="kv_read", s=2, qlo=37, qhi=211, clo=0, chi=30, fmt="int8"),
        # Every token of the decode workload's cache, 64 sequences of up to 8192.
        dict(cache, name="kv_read_all", kind="kv_read", s=64, qlo=512, qhi=8192, clo=0, chi=0, fmt="e4m3"),
        # Four sequences check five proposed tokens each against long contexts: few rows, long keys.
        dict(cache, name="prefill_verify_long", kind="prefill", s=4, qlo=5, qhi=5, clo=8000, chi=32000, fmt="int8", window=0, alibi=False),
        # The chunked-prefill workload over an 8-bit cache: 16 chunks of 512 after up to 7680 tokens.
        dict(cache, name="prefill_chunks", kind="prefill", s=16, qlo=512, qhi=512, clo=0, chi=7680, fmt="e4m3", window=0, alibi=False),
    ]


def _log(rng, lo, hi):
    """A whole number between lo and hi, spread over its logarithm."""
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    kind = rng.choice(["rope", "norm_rope", "norm_rope_bwd", "kv_write", "kv_read", "prefill"])
    d = rng.choice([64, 128])
    hkv = rng.choice([1, 2, 3, 4, 8, 8])
    hq = hkv * rng.choice([1, 2, 4, 4, 5, 8])
    if kind in ("rope", "norm_rope", "norm_rope_bwd"):
        layout = rng.choice(["tokens", "heads"])
        b = 1 if layout == "tokens" else _log(rng, 1, 4)
        n = _log(rng, 1, max(1, (1 << 26) // (b * (hq + hkv) * d)))
        case = dict(kind=kind, layout=layout, b=b, n=n, hq=hq, hkv=hkv, d=d, rot=rng.choice([d, d, d // 2, d // 4, 2 * rng.randint(1, d // 2)]),
                    interleaved=rng.random() < 0.5, dtype=rng.choice(["bf16", "bf16", "f32"]), base=rng.choice([10000.0, 500000.0]),
                    factor=rng.choice([1.0, 1.0, 8.0]), far=_log(rng, 2048, 1 << 20))
        if kind == "rope":
            case["transpose"] = rng.random() < 0.5
        return case
    case = dict(kind=kind, hq=hq, hkv=hkv, d=d, fmt=rng.choice(["e4m3", "int8"]), lengths=rng.randrange(1 << 30))
    if kind == "kv_write":
        q = _log(rng, 1, 2048)
        case.update(s=_log(rng, 1, max(1, min(128, 16384 // q))), qlo=max(0, q // 3), qhi=q, clo=0, chi=_log(rng, 16, 8192))
    elif kind == "kv_read":
        q = _log(rng, 1, 16384)
        case.update(s=_log(rng, 1, max(1, min(128, 131072 // q))), qlo=max(0, q // 4), qhi=q, clo=0, chi=_log(rng, 1, 200))
    else:
        q = _log(rng, 1, 700)
        case.update(s=_log(rng, 1, max(1, min(16, 4096 // q))), qlo=max(0, q // 2), qhi=q, clo=0, chi=_log(rng, 16, 7600),
                    window=rng.choice([0, 0, 0, rng.randint(1, 3000)]), alibi=rng.random() < 0.25)
    return case


# ------------------------------------------------------------- inputs in hand

def _generator(seed):
    return torch.Generator(device=DEV).manual_seed(seed)


def frequencies(rot, base, factor, original=8192):
    """Angles per position of the rot/2 pairs, in 64 bits, and the factor on both functions: plain (factor 1), or
    stretched by parts for contexts `factor` times the original."""
    i = np.arange(rot // 2, dtype=np.float64)
    f = base ** (-2.0 * i / rot)
    if factor == 1.0:
        return f, 1.0
    turns = original * f / (2.0 * math.pi)  # of each pair over the original context
    keep = np.clip((turns - 1.0) / (32.0 - 1.0), 0.0, 1.0)
    return f * keep + f / factor * (1.0 - keep), 0.1 * math.log(factor) + 1.0


def _prepare_rotation(case, seed):
    g = _generator(seed)
    b, n, hq, hkv, d = case["b"], case["n"], case["hq"], case["hkv"], case["d"]
    dt = DTYPES[case["dtype"]]
    f, factor = frequencies(case["rot"], case["base"], case["factor"])
    st = dict(case=case, inv_freq=torch.from_numpy(f).to(DEV), factor=factor)

    def projected():
        """q and k as views of one projection's output, its third part the values."""
        if case["layout"] == "tokens":
            x = torch.randn(n, hq + 2 * hkv, d, generator=g, device=DEV).to(dt)
            return x[:, :hq], x[:, hq:hq + hkv]
        q = torch.randn(b, hq, n, d, generator=g, device=DEV).to(dt)
        return q, torch.randn(b, hkv, n, d, generator=g, device=DEV).to(dt)

    st["q"], st["k"] = projected()
    if case["layout"] == "tokens":  # tokens of many sequences, each at its own place
        st["positions"] = torch.randint(0, case["far"], (n,), generator=g, device=DEV, dtype=torch.int32)
    else:  # each sequence of the batch starts somewhere of its own
        start = torch.randint(0, max(1, case["far"] - n), (b, 1), generator=g, device=DEV, dtype=torch.int32)
        st["positions"] = start + torch.arange(n, device=DEV, dtype=torch.int32)
    if case["kind"] != "rope":
        st["q_weight"] = (1.0 + 0.2 * torch.randn(d, generator=g, device=DEV)).to(dt)
        st["k_weight"] = (1.0 + 0.2 * torch.randn(d, generator=g, device=DEV)).to(dt)
    if case["kind"] == "norm_rope_bwd":
        st["dq_out"], st["dk_out"] = (t.contiguous() for t in projected())
    return st


def _lengths(case):
    """New and earlier tokens of every sequence: the case's own, whatever the seed of the values."""
    r = np.random.RandomState(case["lengths"])
    q = r.randint(case["qlo"], case["qhi"] + 1, case["s"])
    q[0] = case["qhi"]
    c = r.randint(case["clo"], case["chi"] + 1, case["s"])
    return q, c


def _prepare_cache(case, seed):
    g = _generator(seed)
    s, hq, hkv, d, fmt = case["s"], case["hq"], case["hkv"], case["d"], case["fmt"]
    qlens, ctx = _lengths(case)
    lens = qlens + ctx
    blocks = -(-lens // PAGE)
    num_pages, max_blocks = int(blocks.sum()) + 3, max(1, int(blocks.max()))
    perm = torch.randperm(num_pages, generator=torch.Generator().manual_seed(seed)).to(torch.int32).numpy()
    table = np.full((s, max_blocks), -1, dtype=np.int32)
    ends = np.cumsum(blocks)
    for i in range(s):
        table[i, :blocks[i]] = perm[ends[i] - blocks[i]:ends[i]]
    cu = np.concatenate([[0], np.cumsum(qlens)]).astype(np.int32)

    def dev(x):
        return torch.from_numpy(np.ascontiguousarray(x)).to(DEV)

    st = dict(case=case, block_table=dev(table), seq_lens=dev(lens.astype(np.int32)), cu_q=dev(cu), tokens=int(cu[-1]), max_q=int(qlens.max()))
    for name in ("k", "v"):
        # The cache as earlier steps left it: normal values, some channels stronger, each slice at its own scale.
        x = torch.randn(num_pages, hkv, PAGE, d, generator=g, device=DEV)
        x *= torch.exp(0.5 * torch.randn(1, hkv, 1, d, generator=g, device=DEV))
        scales = (x.abs().amax((2, 3)).double() / QMAX[fmt]).float()
        x /= scales[:, :, None, None]
        st[name + "_pages"] = x.round_().clamp_(-127, 127).to(torch.int8) if fmt == "int8" else x.clamp_(-448, 448).to(CODES[fmt])
        st[name + "_scales"] = scales
        del x
    if case["kind"] == "kv_write":
        x = torch.randn(st["tokens"], hq + 2 * hkv, d, generator=g, device=DEV)
        x *= torch.exp(0.5 * torch.randn(1, hq + 2 * hkv, d, generator=g, device=DEV))
        x = x.to(torch.bfloat16)
        st["k"], st["v"] = x[:, hq:hq + hkv], x[:, hq + hkv:]
    if case["kind"] == "prefill":
        st["q"] = torch.randn(st["tokens"], hq, d, generator=g, device=DEV).to(torch.bfloat16)
        st["slopes"] = torch.tensor([2.0 ** (-8.0 * (h + 1) / hq) for h in range(hq)], device=DEV) if case["alibi"] else None
    return st


def prepare(case, seed):
    return (_prepare_rotation if case["kind"] in ("rope", "norm_rope", "norm_rope_bwd") else _prepare_cache)(case, seed)


# ------------------------------------------------------------ the plain forms

def _angles(st):
    """cos and sin of every token and pair, [B or 1, 1, N, rot/2] or [T, 1, rot/2]: the angles in 64 bits, since a far
    position's has no fraction left in 32."""
    a = st["positions"].double()[..., None] * st["inv_freq"]
    a = a.unsqueeze(-2) if st["case"]["layout"] == "tokens" else a.unsqueeze(-3)
    return (torch.cos(a) * st["factor"]).float(), (torch.sin(a) * st["factor"]).float()


def _turn(x, cos, sin, case):
    """The first rot elements of each row turned, pair by pair."""
    r = case["rot"]
    a, b = (x[..., 0:r:2], x[..., 1:r:2]) if case["interleaved"] else (x[..., :r // 2], x[..., r // 2:r])
    y, z = a * cos - b * sin, a * sin + b * cos
    turned = torch.stack((y, z), -1).flatten(-2) if case["interleaved"] else torch.cat((y, z), -1)
    return torch.cat((turned, x[..., r:]), -1)


def _rms(x):
    return torch.rsqrt((x * x).mean(-1, keepdim=True) + 1e-6)


def _plain_rope(st):
    case = st["case"]
    cos, sin = _angles(st)
    sin = -sin if case["transpose"] else sin
    return tuple(_turn(st[n].float(), cos, sin, case).to(st[n].dtype) for n in ("q", "k"))


def _plain_norm_rope(st):
    cos, sin = _angles(st)

    def one(name):
        x = st[name].float()
        return _turn(x * _rms(x) * st[name + "_weight"].float(), cos, sin, st["case"]).to(st[name].dtype)

    return one("q"), one("k")


def _plain_norm_rope_bwd(st):
    cos, sin = _angles(st)

    def one(name):
        x = st[name].float()
        u = _turn(st["d%s_out" % name].float(), cos, -sin, st["case"])
        r = _rms(x)
        h = x * r
        dw = (u * h).flatten(0, -2).sum(0, dtype=torch.float64).float()
        u = u * st[name + "_weight"].float()
        return (r * (u - h * (u * h).mean(-1, keepdim=True))).to(st[name].dtype), dw

    (dq, dqw), (dk, dkw) = one("q"), one("k")
    return dq, dk, dqw, dkw


def _round_code(x, fmt):
    """64-bit quotients to codes, ties to even, kept within the format."""
    if fmt == "int8":
        return x.round().clamp(-127, 127).to(torch.int8)
    # E4M3: 3 bits behind the leading one, steps of 2^-9 below 2^-6.
    step = torch.exp2((torch.frexp(x).exponent - 4).clamp(min=-9).double())
    return ((x / step).round() * step).clamp(-448, 448).float().to(torch.float8_e4m3fn)


def _token_places(st):
    """Sequence, page and slot of every token of the chunks."""
    seq = torch.repeat_interleave(torch.arange(st["case"]["s"], device=DEV), (st["cu_q"][1:] - st["cu_q"][:-1]).long(), output_size=st["tokens"])
    pos = st["seq_lens"][seq].long() - st["cu_q"][seq + 1].long() + torch.arange(st["tokens"], device=DEV)
    return st["block_table"][seq, pos // PAGE].long(), pos % PAGE


def _plain_kv_write(st):
    fmt = st["case"]["fmt"]
    page, slot = _token_places(st)
    # Pages that hold earlier tokens of their sequence: those keep their scale as a floor.
    qlens = st["cu_q"][1:] - st["cu_q"][:-1]
    ctx = st["seq_lens"] - qlens
    shared = (qlens > 0) & (ctx % PAGE > 0)
    last = (ctx // PAGE).clamp(max=st["block_table"].shape[1] - 1).long()
    old_page = torch.where(shared, st["block_table"].gather(1, last[:, None])[:, 0], torch.full_like(ctx, -1)).long()

    def one(x, pages, scales):
        num = pages.shape[0]
        x = x.float()
        amax = torch.zeros(num, pages.shape[1], device=DEV).index_reduce_(0, page, x.abs().amax(-1), "amax")
        new = (amax.double() / torch.full_like(amax, QMAX[fmt], dtype=torch.float64)).float().clamp(min=TINY)
        safe = old_page.clamp(min=0)
        old = scales[safe]
        grown = torch.maximum(old, new[safe])
        new = torch.where(torch.zeros(num, device=DEV).index_add_(0, old_page.clamp(min=0), shared.float())[:, None] > 0,
                          torch.zeros_like(new).index_add_(0, safe, torch.where(shared[:, None], grown, torch.zeros_like(grown))), new)
        # Earlier tokens of those pages, at the new scale.
        codes = pages[safe]
        again = _round_code(codes.double() * old.double()[:, :, None, None] / grown.double()[:, :, None, None], fmt)
        before = (torch.arange(PAGE, device=DEV) < (ctx % PAGE)[:, None]) & shared[:, None]
        kept = torch.where(before[:, None, :, None], again.view(torch.uint8), codes.view(torch.uint8))
        row = torch.where(shared, safe, torch.full_like(safe, num))  # others to a row of no page
        raw = torch.cat((pages.view(torch.uint8), torch.zeros_like(pages[:1].view(torch.uint8))))
        raw[row] = kept
        raw[page, :, slot] = _round_code(x.double() / new.double()[page][:, :, None], fmt).view(torch.uint8)
        pages.view(torch.uint8).copy_(raw[:num])
        scales[page] = new[page]

    one(st["k"], st["k_pages"], st["k_scales"])
    one(st["v"], st["v_pages"], st["v_scales"])
    return st["k_pages"], st["v_pages"], st["k_scales"], st["v_scales"]


def _plain_kv_read(st):
    page, slot = _token_places(st)
    return tuple((st[n + "_pages"].view(torch.uint8)[page, :, slot].view(CODES[st["case"]["fmt"]]).float() * st[n + "_scales"][page][:, :, None]).to(torch.bfloat16)
                 for n in ("k", "v"))


def _plain_prefill(st):
    case = st["case"]
    s, hq, hkv, d, t = case["s"], case["hq"], case["hkv"], case["d"], st["tokens"]
    table = st["block_table"].clamp(min=0).long()
    keys = table.shape[1] * PAGE

    def dense(n):  # [S, Hkv, 1, keys, d]
        x = st[n + "_pages"].view(torch.uint8)[table].view(CODES[case["fmt"]]).float() * st[n + "_scales"][table][..., None, None]
        return x.transpose(1, 2).reshape(s, hkv, 1, keys, d)

    qlens = (st["cu_q"][1:] - st["cu_q"][:-1]).long()
    seq = torch.repeat_interleave(torch.arange(s, device=DEV), qlens, output_size=t)
    at = torch.arange(t, device=DEV) - st["cu_q"][seq].long()
    q = torch.zeros(s, st["max_q"], hq, d, device=DEV)
    q[seq, at] = st["q"].float()
    q = q.transpose(1, 2).reshape(s, hkv, hq // hkv, st["max_q"], d)
    x = torch.matmul(q, dense("k").transpose(-1, -2)).mul_(1.0 / math.sqrt(d))
    pos = (st["seq_lens"].long() - qlens)[:, None] + torch.arange(st["max_q"], device=DEV)  # [S, max_q]
    back = pos[:, :, None] - torch.arange(keys, device=DEV)  # how far behind the query a key lies
    seen = (back >= 0) & (back < case["window"]) if case["window"] else back >= 0
    if st["slopes"] is not None:
        x -= st["slopes"].view(1, hkv, hq // hkv, 1, 1) * back[:, None, None].float()
    x.masked_fill_(~seen[:, None, None], -math.inf)
    m = x.amax(-1, keepdim=True)
    x.sub_(m).exp_()
    l = x.sum(-1, keepdim=True)
    o = torch.matmul(x, dense("v")) / l
    o = o.reshape(s, hq, st["max_q"], d).transpose(1, 2)[seq, at].to(torch.bfloat16)
    lse = (m + torch.log(l)).reshape(s, hq, st["max_q"]).transpose(1, 2)[seq, at]
    return o, lse


_PLAIN = dict(rope=_plain_rope, norm_rope=_plain_norm_rope, norm_rope_bwd=_plain_norm_rope_bwd, kv_write=_plain_kv_write, kv_read=_plain_kv_read,
              prefill=_plain_prefill)


# --------------------------------------------------------- the library's calls

def _own(st):
    import exact_io_aware_101_b200 as ea

    case = st["case"]
    kind = case["kind"]
    if kind in ("rope", "norm_rope", "norm_rope_bwd"):
        how = dict(interleaved=case["interleaved"], attention_factor=st["factor"])
        if kind == "rope":
            return ea.attn_rope(st["q"], st["k"], st["positions"], st["inv_freq"], transpose=case["transpose"], **how)
        if kind == "norm_rope":
            return ea.attn_norm_rope(st["q"], st["k"], st["q_weight"], st["k_weight"], st["positions"], st["inv_freq"], eps=1e-6, **how)
        return ea.attn_norm_rope_bwd(st["q"], st["k"], st["q_weight"], st["k_weight"], st["dq_out"], st["dk_out"], st["positions"], st["inv_freq"],
                                     eps=1e-6, **how)
    cache = (st["k_pages"], st["v_pages"], st["k_scales"], st["v_scales"], st["block_table"], st["seq_lens"], st["cu_q"])
    if kind == "kv_write":
        ea.attn_kv_write_paged_q8(st["k"], st["v"], *cache, max_q=st["max_q"], kv_format=case["fmt"])
        return st["k_pages"], st["v_pages"], st["k_scales"], st["v_scales"]
    if kind == "kv_read":
        return ea.attn_kv_read_paged_q8(*cache, tokens=st["tokens"], max_q=st["max_q"], kv_format=case["fmt"])
    return ea.attn_prefill_paged_q8(st["q"], *cache, max_q=st["max_q"], kv_format=case["fmt"], window=case["window"], alibi_slopes=st["slopes"])


def run(state):
    if own:
        return _own(state)
    return _PLAIN[state["case"]["kind"]](state)


# ------------------------------------------------------------------- the work

def work(case):
    """Bytes: each input read once, each output written once."""
    d, hq, hkv = case["d"], case["hq"], case["hkv"]
    if case["kind"] in ("rope", "norm_rope", "norm_rope_bwd"):
        rows = case["b"] * case["n"] * (hq + hkv)
        size = 2 if case["dtype"] == "bf16" else 4
        passes = 3 if case["kind"] == "norm_rope_bwd" else 2
        flops = {"rope": 3 * case["rot"], "norm_rope": 4 * d + 3 * case["rot"], "norm_rope_bwd": 10 * d + 3 * case["rot"]}[case["kind"]]
        return {"bytes": passes * rows * d * size + 4 * case["b"] * case["n"] + 8 * (case["rot"] // 2), "flops": rows * flops}
    q, c = (x.astype(np.int64) for x in _lengths(case))
    tokens, row = int(q.sum()), 2 * hkv * d  # elements of a token's keys and values
    table = 4 * (2 * len(q) + 1)
    if case["kind"] in ("kv_write", "kv_read"):
        pages = int((-(-(q + c) // PAGE) - c // PAGE)[q > 0].sum())
        if case["kind"] == "kv_read":
            return {"bytes": tokens * row * 3 + pages * (4 + 8 * hkv) + table, "flops": tokens * row}
        return {"bytes": tokens * row * 3 + pages * (4 + 8 * hkv) + table, "flops": tokens * row * 3}
    seen = q * c + q * (q + 1) // 2
    keys = np.where(q > 0, q + c, 0)
    if case["window"]:
        w = case["window"]
        first = np.minimum(np.maximum(w - c, 0), q)  # the queries that see every key behind them
        seen = first * c + first * (first + 1) // 2 + (q - first) * w
        keys = np.where(q > 0, np.minimum(keys, q + w - 1), 0)
    pages = int((-(-keys // PAGE)).sum())
    return {"bytes": tokens * hq * (4 * d + 4) + int(keys.sum()) * row + pages * (4 + 8 * hkv) + table, "flops": 4 * d * hq * int(seen.sum())}


# -------------------------------------------------- the definition, in 64 bits

def _rotation_matrix_product(x, angle, factor, case):
    """Each pair of elements (of the first rot) as a complex number times factor * exp(i angle)."""
    r, y = case["rot"], x.clone()
    first = slice(0, r, 2) if case["interleaved"] else slice(0, r // 2)
    second = slice(1, r, 2) if case["interleaved"] else slice(r // 2, r)
    z = torch.complex(x[..., first].contiguous(), x[..., second].contiguous()) * torch.polar(torch.full_like(angle, factor), angle)
    y[..., first], y[..., second] = z.real, z.imag
    return y


def _exact_rotation(st):
    case = st["case"]
    angle = st["positions"].double()[..., None] * st["inv_freq"]
    angle = angle[:, None] if case["layout"] == "tokens" else angle[:, None, :, :]
    out = []
    for name in ("q", "k"):
        x = st[name].double()
        if case["kind"] == "rope":
            out.append(_rotation_matrix_product(x, -angle if case["transpose"] else angle, st["factor"], case))
            continue
        w = st[name + "_weight"].double()
        if case["kind"] == "norm_rope":
            out.append(_rotation_matrix_product(x / torch.sqrt((x ** 2).sum(-1, keepdim=True) / case["d"] + 1e-6) * w, angle, st["factor"], case))
            continue
        x.requires_grad_(True)
        w.requires_grad_(True)
        # The gradient by differentiation: of sum(dy * R(angle) y) = sum((R(-angle) dy) * y).
        u = _rotation_matrix_product(st["d%s_out" % name].double(), -angle, st["factor"], case)
        y = x / torch.sqrt((x ** 2).sum(-1, keepdim=True) / case["d"] + 1e-6) * w
        out.append(torch.autograd.grad((y * u).sum(), (x, w)))
    if case["kind"] == "norm_rope_bwd":
        return out[0][0], out[1][0], out[0][1], out[1][1]
    return tuple(out)


def _nearest_codes(x, fmt):
    """The format's values nearest to x (64 bits), ties to the even code: by search in the sorted list of values."""
    if fmt == "int8":
        values = torch.arange(-127, 128, dtype=torch.float64, device=DEV)
        even = torch.arange(-127, 128, device=DEV) % 2 == 0
    else:
        codes = torch.arange(0, 127, dtype=torch.uint8, device=DEV)
        mag = codes.view(torch.float8_e4m3fn).double()
        values = torch.cat((-mag.flip(0)[:-1], mag))
        even = torch.cat(((codes % 2 == 0).flip(0)[:-1], codes % 2 == 0))
    hi = torch.searchsorted(values, x.contiguous()).clamp(1, len(values) - 1)
    lo = hi - 1
    up, down = values[hi] - x, x - values[lo]
    return values[torch.where((up < down) | ((up == down) & even[hi]), hi, lo)]


def _exact_kv_write(st):
    case, out = st["case"], []
    cu, lens, table = st["cu_q"].tolist(), st["seq_lens"].tolist(), st["block_table"].tolist()
    jobs = []  # (page, slots kept, first token, tokens)
    for i in range(case["s"]):
        t, pos = cu[i], lens[i] - (cu[i + 1] - cu[i])
        while t < cu[i + 1]:
            n = min(PAGE - pos % PAGE, cu[i + 1] - t)
            jobs.append((table[i][pos // PAGE], pos % PAGE, t, n))
            t, pos = t + n, pos + n
    for name in ("k", "v"):
        codes, scales = st[name + "_pages"].double(), st[name + "_scales"].double()
        x = st[name].double()
        if len(jobs) <= 6000:
            for page, kept, t, n in jobs:
                rows = x[t:t + n].transpose(0, 1)  # [Hkv, n, d]
                sc = (rows.abs().amax((1, 2)) / QMAX[case["fmt"]]).float().double().clamp(min=TINY)
                if kept:
                    sc = torch.maximum(sc, scales[page])
                    codes[page, :, :kept] = _nearest_codes(codes[page, :, :kept] * scales[page][:, None, None] / sc[:, None, None], case["fmt"])
                codes[page, :, kept:kept + n] = _nearest_codes(rows / sc[:, None, None], case["fmt"])
                scales[page] = sc
            out.append((codes.to(torch.int8) if case["fmt"] == "int8" else codes, scales))
        else:
            return None
    return out[0][0], out[1][0], out[0][1], out[1][1]


def _sequence(st, name, i, n):
    """The n tokens of sequence i out of the pages, [n, Hkv, d] in 64 bits."""
    pages = st["block_table"][i, :-(-n // PAGE)].long()
    x = st[name + "_pages"].view(torch.uint8)[pages].view(CODES[st["case"]["fmt"]]).double() * st[name + "_scales"][pages].double()[:, :, None, None]
    return x.transpose(1, 2).flatten(0, 1)[:n]


def _exact_kv_read(st):
    cu, lens = st["cu_q"].tolist(), st["seq_lens"].tolist()
    return tuple(torch.cat([_sequence(st, name, i, n)[n - (cu[i + 1] - cu[i]):] for i, n in enumerate(lens)]) for name in ("k", "v"))


def _exact_prefill(st):
    case = st["case"]
    cu, lens, group = st["cu_q"].tolist(), st["seq_lens"].tolist(), case["hq"] // case["hkv"]
    o = torch.zeros(st["tokens"], case["hq"], case["d"], dtype=torch.float64, device=DEV)
    lse = torch.zeros(st["tokens"], case["hq"], dtype=torch.float64, device=DEV)
    for i, n in enumerate(lens):
        nq = cu[i + 1] - cu[i]
        if not nq:
            continue
        k, v = _sequence(st, "k", i, n), _sequence(st, "v", i, n)
        query, key = torch.arange(n - nq, n, device=DEV)[:, None], torch.arange(n, device=DEV)[None]
        hidden = key > query
        if case["window"]:
            hidden |= key <= query - case["window"]
        for h in range(case["hq"]):
            x = st["q"][cu[i]:cu[i + 1], h].double() @ k[:, h // group].T / math.sqrt(case["d"])
            if st["slopes"] is not None:
                x += st["slopes"][h].double() * (key - query)
            x[hidden] = -math.inf
            lse[cu[i]:cu[i + 1], h] = torch.logsumexp(x, 1)
            o[cu[i]:cu[i + 1], h] = torch.softmax(x, 1) @ v[:, h // group]
    return o, lse


def exact(case, seed):
    st = prepare(case, seed)
    if case["kind"] in ("rope", "norm_rope", "norm_rope_bwd"):
        return _exact_rotation(st)
    return dict(kv_write=_exact_kv_write, kv_read=_exact_kv_read, prefill=_exact_prefill)[case["kind"]](st)
