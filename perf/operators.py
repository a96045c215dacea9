"""The paged-cache operators' cases: what each call does, on which sizes, and what it has to move.

Three operators serve ragged batches over the page pools that fa_decode_paged reads:

  append   new keys and values are written into the pools' pages (quantized where a pool is q4_0);
           a pool in the dtype is returned as it stands, q4_0 pages as the values of the tokens
           just written, read back through the read operator
  read     the last tokens of every sequence, gathered from the pages into packed rows
  prefill  causal attention of every sequence's new tokens over its pages

Packed rows: sequence b owns rows starts[b] .. starts[b + 1] - 1 of the [T, heads, D] tensors, which
are its last tokens, at positions lens[b] - n .. lens[b] - 1.  ``run`` computes the plain form in f32
with elementary torch operations, or calls the library where ``own`` is set.
"""
import math

import torch

own = False  # set by the tools: True calls the library, False computes the plain form

_DTYPES = {"f16": torch.float16, "bf16": torch.bfloat16}


# ------------------------------------------------------------------------------------------
# cases
# ------------------------------------------------------------------------------------------

def _case(name, op, new, ctx, *, dtype="f16", kf="dense", vf="dense", hq=32, hkv=8, d=128,
          page=128, fused=False, pad=0):
    """new: tokens of each sequence in this call; ctx: tokens it already holds in the pages."""
    c = {"op": op, "dtype": dtype, "kf": kf, "vf": vf, "hq": hq, "hkv": hkv, "d": d, "page": page,
         "new": ",".join(map(str, new)), "ctx": ",".join(map(str, ctx)), "fused": fused, "pad": pad}
    return {"name": name, **c} if name else c


def listed():
    q4 = {"kf": "q4_0", "vf": "q4_0"}
    return [
        # a short chat: four users, one new token each, a few hundred tokens of context
        _case("prefill_step_b4_f16", "prefill", [1] * 4, [776, 130, 64, 512], page=64),
        # sixteen users whose draft tokens are verified: five new tokens each over a q4_0 cache
        _case("prefill_drafts_b16_q4_0", "prefill", [5] * 16,
              [4091 - 97 * i for i in range(16)], **q4),
        # continuous batching: fifteen users decode while a 512-token chunk of a sixteenth's prompt
        # joins, in a batch padded to a fixed row count, q cut out of a fused projection, 16-token pages
        _case("prefill_mixed_b16_bf16", "prefill", [1] * 9 + [512] + [1] * 6,
              [250 * i + 33 for i in range(9)] + [1500] + [3000 + 150 * i for i in range(6)],
              dtype="bf16", page=16, fused=True, pad=24),
        # whole prompts of odd lengths at head dim 64, f16 keys with q4_0 values
        _case("prefill_prompts_d64_f16k_q4_0v", "prefill", [333, 1, 1021, 77, 600], [0] * 5,
              hq=8, hkv=8, d=64, vf="q4_0"),
        # the benchmark's chunk: 2048 tokens at the end of 16384, dense and q4_0 caches
        _case("prefill_chunk_sk16384_f16", "prefill", [2048], [14336], page=256),
        _case("prefill_chunk_sk16384_q4_0", "prefill", [2048], [14336], page=256, **q4),
        # one decode step of 64 users written into a q4_0 cache
        _case("append_step_b64_q4_0", "append", [1] * 64, [31 * i + 5 for i in range(64)], **q4),
        # a ragged step into dense 16-token pages, k and v cut out of a fused projection
        _case("append_ragged_b7_bf16", "append", [700, 1, 0, 257, 16, 1, 33],
              [1000, 15, 9, 0, 16, 4000, 255], dtype="bf16", page=16, fused=True, pad=8),
        # four prompt chunks written into a q4_0 cache
        _case("append_chunk_b4_q4_0_bf16", "append", [2048] * 4, [2048 * i for i in range(4)],
              dtype="bf16", page=256, **q4),
        # a few short sequences taken out of the cache
        _case("read_short_b4_q4_0", "read", [129, 1, 640, 57], [0] * 4, **q4),
        # four long sequences taken out of the cache (moved to another worker), dense and q4_0
        _case("read_long_b4_sk16384_f16", "read", [16384] * 4, [0] * 4, page=256),
        _case("read_long_b4_sk16384_q4_0", "read", [16384] * 4, [0] * 4, page=256, **q4),
    ]


def _log_int(rng, lo, hi):
    return min(hi, int(math.exp(rng.uniform(math.log(lo), math.log(hi + 1)))))


def draw(rng):
    while True:
        op = rng.choice(["prefill", "prefill", "append", "read"])
        hq, hkv = rng.choice([(32, 8), (8, 8), (8, 2), (16, 2), (12, 4), (8, 1), (32, 4)])
        n = _log_int(rng, 1, 64)
        top = _log_int(rng, 1, 16384 if op == "read" else 2048)
        new = [_log_int(rng, 1 + top // 8, top) for _ in range(n)]
        if rng.random() < 0.2:
            new = [1] * n  # a decode step
        most = 0 if op == "read" else _log_int(rng, 1, 14336)
        ctx = [_log_int(rng, 1 + most // 8, most) if most and rng.random() < 0.9 else 0
               for _ in range(n)]
        if op == "append" and n > 1:
            new[rng.randrange(n)] = 0  # a sequence with nothing new in this step
        c = _case(None, op, new, ctx, dtype=rng.choice(["f16", "bf16"]),
                  kf=rng.choice(["dense", "q4_0"]), vf=rng.choice(["dense", "q4_0"]), hq=hq,
                  hkv=hkv, d=rng.choice([64, 128]), page=rng.choice([16, 32, 48, 64, 128, 256]),
                  fused=rng.random() < 0.3, pad=rng.choice([0, 0, 1, 40]))
        total = [a + b for a, b in zip(new, ctx)]
        w = work(c)
        # no dearer than the largest listed case, in the plain form's padded scores too
        if (w["bytes"] < 5.3e8 and w["flops"] < 5.1e11 and n * max(total) * hkv * c["d"] < 7e7
                and (op != "prefill" or n * max(new) * hq * max(total) < 1.1e9)):
            return c


def _sizes(case):
    new = [int(x) for x in case["new"].split(",")]
    ctx = [int(x) for x in case["ctx"].split(",")]
    return new, [a + b for a, b in zip(new, ctx)]


def work(case):
    new, lens = _sizes(case)
    hq, hkv, d = case["hq"], case["hkv"], case["d"]
    row = {"dense": 2 * d, "q4_0": d // 2 + d // 16}  # bytes of one head's token in the pages
    cache = hkv * (row[case["kf"]] + row[case["vf"]])
    dense = hkv * 4 * d  # k and v of one token in the dtype
    n = sum(new)
    if case["op"] == "append":
        back = n * dense if "q4_0" in (case["kf"], case["vf"]) else 0  # what is read back
        return {"bytes": n * (dense + cache) + back, "flops": 0}
    if case["op"] == "read":
        return {"bytes": n * (cache + dense), "flops": 0}
    pairs = sum(n_ * l_ - n_ * (n_ - 1) // 2 for n_, l_ in zip(new, lens))
    used = sum(l_ for n_, l_ in zip(new, lens) if n_)
    return {"bytes": used * cache + n * hq * d * 4, "flops": 4 * d * hq * pairs}


# ------------------------------------------------------------------------------------------
# inputs
# ------------------------------------------------------------------------------------------

def _q4_planes(x):
    """q4_0 blocks of 32 along the last axis: (nibbles uint8 [..., D/2], scales f16 [..., D/32]).
    m = the first element of largest magnitude, d = m / -8, code = min(15, trunc(x * (1/d) + 8.5))
    in f32, one rounding a step; element j in byte j's low nibble, j + 16 in its high one."""
    b = x.float().unflatten(-1, (-1, 32))
    mag = b.abs()
    first = (mag == mag.amax(-1, keepdim=True)).to(torch.int8).argmax(-1, keepdim=True)
    d = b.gather(-1, first) / -8.0
    inv = torch.where(d != 0, 1.0 / d, torch.zeros_like(d))
    code = ((b * inv) + 8.5).clamp(0, 15).to(torch.uint8)
    return (code[..., :16] | (code[..., 16:] << 4)).flatten(-2), d.squeeze(-1).to(torch.float16)


def _planes_of(buf, shape):
    """Views of a q4_0 buffer's nibble and scale planes for a pool [N, Hkv, page, D]."""
    n, h, s, d = shape
    nib = n * h * s * d // 2
    off = (nib + 255) // 256 * 256
    return (buf[:nib].view(n, h, s, d // 2),
            buf[off:off + n * h * s * (d // 16)].view(torch.float16).view(n, h, s, d // 32))


def _pool(fmt, shape, dtype, gen):
    x = torch.randn(shape, generator=gen, device="cuda", dtype=torch.float32).to(dtype)
    if fmt == "dense":
        return x
    nib, scale = _q4_planes(x)
    off = (nib.numel() + 255) // 256 * 256
    buf = torch.zeros(off + 2 * scale.numel(), dtype=torch.uint8, device="cuda")
    at, sc = _planes_of(buf, shape)
    at.copy_(nib)
    sc.copy_(scale)
    return buf


def prepare(case, seed):
    new, lens = _sizes(case)
    dt, hq, hkv, d, page = (_DTYPES[case["dtype"]], case["hq"], case["hkv"], case["d"],
                            case["page"])
    gen = torch.Generator(device="cuda").manual_seed(int(seed))
    per_seq = [-(-l_ // page) for l_ in lens]
    pps = max(1, max(per_seq))
    shape = (sum(per_seq) + 2, hkv, page, d)
    perm = torch.randperm(shape[0], generator=gen, device="cuda").to(torch.int32)
    first = [sum(per_seq[:i]) for i in range(len(lens))]
    slot = (torch.tensor(first, device="cuda")[:, None] + torch.arange(pps, device="cuda"))
    held = torch.arange(pps, device="cuda")[None] < torch.tensor(per_seq, device="cuda")[:, None]
    table = torch.where(held, perm[slot.clamp(max=shape[0] - 1)], 0).to(torch.int32).contiguous()
    starts = torch.tensor([sum(new[:i]) for i in range(len(new) + 1)], dtype=torch.int32,
                          device="cuda")
    rows = sum(new) + case["pad"]
    s = {"case": case, "dt": dt, "shape": shape, "table": table, "starts": starts,
         "lens": torch.tensor(lens, dtype=torch.int32, device="cuda"),
         "k_pages": _pool(case["kf"], shape, dt, gen), "v_pages": _pool(case["vf"], shape, dt, gen),
         "n": sum(new), "max_new": max(new)}

    def packed(*heads):
        """Packed rows for each of `heads`, cut out of one fused tensor where the case says so."""
        if case["fused"]:
            x = torch.randn(rows, sum(heads), d, generator=gen, device="cuda").to(dt)
            return torch.split(x, heads, dim=1)
        return [torch.randn(rows, h, d, generator=gen, device="cuda").to(dt) for h in heads]

    if case["op"] == "prefill":
        s["q"] = packed(hq, hkv, hkv)[0] if case["fused"] else packed(hq)[0]
        s["o"] = torch.zeros(rows, hq, d, dtype=dt, device="cuda")
    else:
        if case["op"] == "append":
            s["k_new"], s["v_new"] = packed(hq, hkv, hkv)[1:] if case["fused"] else packed(hkv, hkv)
        s["k_out"] = torch.zeros(rows, hkv, d, dtype=dt, device="cuda")
        s["v_out"] = torch.zeros(rows, hkv, d, dtype=dt, device="cuda")
    return s


# ------------------------------------------------------------------------------------------
# one pass
# ------------------------------------------------------------------------------------------

def _values(pages, fmt, shape):
    """A pool's values in f32."""
    if fmt == "dense":
        return pages.float()
    nib, scale = _planes_of(pages, shape)
    b = nib.unflatten(-1, (-1, 16))
    code = torch.cat((b & 15, b >> 4), -1).float() - 8.0
    return (code * scale.float()[..., None]).flatten(-2)


def _tokens(s):
    """For every packed row that belongs to a sequence: its sequence, its place in the sequence's
    rows, its page and its slot in the page."""
    row = torch.arange(s["n"], device="cuda")
    b = (row[:, None] >= s["starts"][None, 1:]).sum(1)
    i = row - s["starts"][b]
    pos = i + s["lens"][b] - (s["starts"][b + 1] - s["starts"][b])
    page = s["case"]["page"]
    return b, i, s["table"][b, pos // page].long(), pos % page


def _plain_read(s, pages, fmt, out):
    _, _, page, slot = _tokens(s)
    if fmt == "dense":
        got = pages[page, :, slot]
    else:
        nib, scale = _planes_of(pages, s["shape"])
        b = nib[page, :, slot].unflatten(-1, (-1, 16))
        code = torch.cat((b & 15, b >> 4), -1).float() - 8.0
        got = (code * scale[page, :, slot].float()[..., None]).flatten(-2)
    out[:s["n"]] = got.to(out.dtype)
    return out


def _plain_write(s, x, pages, fmt):
    _, _, page, slot = _tokens(s)
    if fmt == "dense":
        pages[page, :, slot] = x[:s["n"]]
    else:
        nib, scale = _planes_of(pages, s["shape"])
        n, sc = _q4_planes(x[:s["n"]])
        nib[page, :, slot] = n
        scale[page, :, slot] = sc


def _plain_prefill(s):
    c = s["case"]
    hq, hkv, d, g = c["hq"], c["hkv"], c["d"], c["hq"] // c["hkv"]
    table, lens, starts = s["table"].long(), s["lens"], s["starts"]
    n_b, cap = len(lens), s["table"].shape[1] * c["page"]
    key = torch.arange(cap, device="cuda")
    held = key[None] < lens[:, None]

    def gathered(name, fmt):  # [B, Hkv, cap, D] f32, zero past each sequence's end
        x = _values(s[name], fmt, s["shape"])[table].permute(0, 2, 1, 3, 4).flatten(2, 3)
        return torch.where(held[:, None, :, None], x, 0.0)

    m = s["max_new"]
    i = torch.arange(m, device="cuda")
    rows = (starts[:-1, None] + i[None]).clamp(max=s["q"].shape[0] - 1)
    q = s["q"].float()[rows].permute(0, 2, 1, 3).reshape(n_b, hkv, g * m, d)  # rows: head, token
    p = torch.matmul(q, gathered("k_pages", c["kf"]).transpose(-1, -2)).mul_(d ** -0.5)
    pos = lens[:, None] - (starts[1:] - starts[:-1])[:, None] + i[None]
    sees = (key[None, None] <= pos[:, :, None]) & held[:, None]  # [B, m, cap]
    p = p.view(n_b, hkv, g, m, cap)
    p.masked_fill_(~sees[:, None, None], -math.inf)
    top = p.amax(-1, keepdim=True)
    p.sub_(torch.where(top == -math.inf, 0.0, top)).exp_()
    total = p.sum(-1, keepdim=True)
    o = torch.matmul(p.view(n_b, hkv, g * m, cap), gathered("v_pages", c["vf"]))
    o = o.view(n_b, hkv, g, m, d) / torch.where(total == 0, 1.0, total)
    b, at, _, _ = _tokens(s)
    s["o"][:s["n"]] = o.permute(0, 3, 1, 2, 4).reshape(n_b, m, hq, d)[b, at].to(s["dt"])
    return s["o"]


def _wrapped(s, name, fmt):
    import quantized_kv_cache_sm_gb300 as fa

    return s[name] if fmt == "dense" else fa.Q4Tensor(s[name], *s["shape"])


def _own(s):
    import quantized_kv_cache_sm_gb300 as fa

    c = s["case"]
    k, v = _wrapped(s, "k_pages", c["kf"]), _wrapped(s, "v_pages", c["vf"])
    batch = (s["table"], s["starts"], s["lens"])
    if c["op"] == "prefill":
        return fa.fa_prefill_paged(s["q"], k, v, *batch, s["o"])
    if c["op"] == "append":
        fa.fa_append_paged(s["k_new"], s["v_new"], k, v, *batch)
        if "q4_0" not in (c["kf"], c["vf"]):
            return s["k_pages"], s["v_pages"]
    return fa.fa_read_paged(k, v, *batch, s["k_out"], s["v_out"])


def run(state):
    if own:
        return _own(state)
    c = state["case"]
    if c["op"] == "prefill":
        return _plain_prefill(state)
    if c["op"] == "append":
        _plain_write(state, state["k_new"], state["k_pages"], c["kf"])
        _plain_write(state, state["v_new"], state["v_pages"], c["vf"])
        if "q4_0" not in (c["kf"], c["vf"]):
            return state["k_pages"], state["v_pages"]
    return (_plain_read(state, state["k_pages"], c["kf"], state["k_out"]),
            _plain_read(state, state["v_pages"], c["vf"], state["v_out"]))


# ------------------------------------------------------------------------------------------
# the same in 64 bits, sequence by sequence
# ------------------------------------------------------------------------------------------

def _exact_sequence(s, name, fmt, b, length):
    """[Hkv, length, D] f64: sequence b's tokens in order."""
    page = s["case"]["page"]
    ids = s["table"][b, :-(-length // page)].long()
    if fmt == "dense":
        x = s[name][ids].double()
    else:
        nib, scale = (p[ids] for p in _planes_of(s[name], s["shape"]))
        n, h, p, w = nib.shape
        code = torch.empty(n, h, p, w // 16, 32, dtype=torch.float64, device="cuda")
        code[..., :16] = nib.view(n, h, p, w // 16, 16) % 16
        code[..., 16:] = nib.view(n, h, p, w // 16, 16) // 16
        x = ((code - 8.0) * scale.double()[..., None]).view(n, h, p, 2 * w)
    return x.transpose(0, 1).reshape(x.shape[1], -1, x.shape[-1])[:, :length]


def _exact_q4(x):
    """The values that q4_0 blocks of x stand for, in f64."""
    b = x.double().unflatten(-1, (-1, 32))
    m = b.gather(-1, b.abs().max(-1, keepdim=True).indices)
    d = m / -8.0
    code = torch.where(d == 0, torch.full_like(b, 8.0),
                       torch.floor(b / torch.where(d == 0, torch.ones_like(d), d) + 8.5))
    return ((code.clamp(0, 15) - 8.0) * d.to(torch.float16).double()).flatten(-2)


def exact(case, seed):
    s = prepare(case, seed)
    new, lens = _sizes(case)
    rows = s["n"] + case["pad"]
    if case["op"] == "prefill":
        g, d = case["hq"] // case["hkv"], case["d"]
        o = torch.zeros(rows, case["hq"], d, dtype=torch.float64, device="cuda")
        at = 0
        for b, (n, length) in enumerate(zip(new, lens)):
            if n == 0:
                continue
            k = _exact_sequence(s, "k_pages", case["kf"], b, length)
            v = _exact_sequence(s, "v_pages", case["vf"], b, length)
            hidden = (torch.arange(length, device="cuda")[None]
                      > torch.arange(length - n, length, device="cuda")[:, None])
            for h in range(case["hq"]):
                t = (s["q"][at:at + n, h].double() @ k[h // g].T) / math.sqrt(d)
                w = torch.softmax(t.masked_fill(hidden, -math.inf), -1)
                o[at:at + n, h] = w @ v[h // g]
            at += n
        return o
    if case["op"] == "append" and "q4_0" not in (case["kf"], case["vf"]):
        pools = (s["k_pages"].double(), s["v_pages"].double())
        at = 0
        for b, (n, length) in enumerate(zip(new, lens)):
            pos = torch.arange(length - n, length, device="cuda")
            where = s["table"][b, pos // case["page"]].long()
            for pool, x in zip(pools, (s["k_new"], s["v_new"])):
                pool[where, :, pos % case["page"]] = x[at:at + n].double()
            at += n
        return pools
    out = []
    for name, fmt in (("k", case["kf"]), ("v", case["vf"])):
        o = torch.zeros(rows, case["hkv"], case["d"], dtype=torch.float64, device="cuda")
        if case["op"] == "append":
            x = s[name + "_new"][:s["n"]]
            o[:s["n"]] = _exact_q4(x) if fmt == "q4_0" else x.double()
        else:
            at = 0
            for b, (n, length) in enumerate(zip(new, lens)):
                o[at:at + n] = _exact_sequence(s, name + "_pages", fmt, b,
                                               length)[:, length - n:].transpose(0, 1)
                at += n
        out.append(o)
    return tuple(out)
