"""The serving operators of the quantized layer and its key/value cache, as they are measured.

Four operators that one decoding step of an attention block runs together:

* decode: y = x W_Q^T + alpha z F^T for the few tokens of a decoding step (qwha_layer_decode);
* write:  new keys and values quantized into a paged cache, and read back (qwha_cache_write and
  qwha_cache_read of the same slots: what is stored is compared as the values it stands for);
* read:   cached tokens read back as dense keys and values (qwha_cache_read);
* attn:   attention of one query token per sequence over the paged cache (qwha_cache_attn).

`run` computes them in elementary torch operations, or, where `own` is set, through the library.
"""
import math

import torch

own = False

DEV = "cuda:0"
DTYPES = {"bf16": torch.bfloat16, "f32": torch.float32}


# ---------------------------------------------------------------- the cases
def listed():
    return [
        # the smallest layer, one fp32 token: nothing but latency
        dict(name="decode_256_t1_f32", op="decode", act="f32", T=1, d_out=256, d_in=256, bits=4,
             group=64, p=2048),
        # the q or o projection of an attention block, one sequence being decoded
        dict(name="decode_4096_t1", op="decode", act="bf16", T=1, d_out=4096, d_in=4096, bits=4,
             group=128, p=524288),
        # the down projection (block-diagonal transform), a handful of sequences
        dict(name="decode_4096x14336_t3", op="decode", act="bf16", T=3, d_out=4096, d_in=14336,
             bits=4, group=128, p=1179648),
        # the gate or up projection at 3 bits, a batch of sixteen sequences
        dict(name="decode_14336x4096_t16", op="decode", act="bf16", T=16, d_out=14336, d_in=4096,
             bits=3, group=128, p=1179648),
        # a wide layer at 2 bits and small groups, the largest batch of a decoding step
        dict(name="decode_8192_t64", op="decode", act="bf16", T=64, d_out=8192, d_in=8192, bits=2,
             group=64, p=1048576),
        # one decoding step of 32 sequences: 8 key/value heads of 128
        dict(name="write_32", op="write", act="bf16", T=32, heads=8, dim=128, page=16, pages=1024,
             bits=4, rotate=True),
        # a prompt written at once
        dict(name="write_8192", op="write", act="bf16", T=8192, heads=8, dim=128, page=64,
             pages=256, bits=4, rotate=True),
        # one sequence of odd length, 8-bit codes without the transform, fp32 output
        dict(name="read_1001_f32", op="read", act="f32", T=1001, heads=4, dim=64, page=16, pages=80,
             bits=8, rotate=False),
        # a long context read back for a prompt's next chunk
        dict(name="read_40000", op="read", act="bf16", T=40000, heads=8, dim=128, page=64,
             pages=700, bits=4, rotate=True),
        # one short sequence: latency
        dict(name="attn_b1_777", op="attn", act="bf16", B=1, kv_heads=8, per_kv=4, dim=128, page=16,
             len=777, shortest=777, bits=4, rotate=True),
        # a full batch of ragged lengths
        dict(name="attn_b32_4096", op="attn", act="bf16", B=32, kv_heads=8, per_kv=4, dim=128,
             page=64, len=4096, shortest=1900, bits=4, rotate=True),
        # long contexts, as many key heads as query heads, 8-bit codes, fp32 queries, one
        # sequence without any token yet
        dict(name="attn_b3_30001_f32", op="attn", act="f32", B=3, kv_heads=16, per_kv=1, dim=64,
             page=32, len=30001, shortest=0, bits=8, rotate=False),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def _cost(case):
    w = work(case)
    return max(w["bytes"], w["flops"] / 50)


def _drawn(rng):
    op = rng.choice(["decode", "decode", "write", "read", "attn", "attn"])
    act = rng.choice(["bf16", "bf16", "f32"])
    if op == "decode":
        # every multiple of 64 has a transform
        d_in = 64 * _log(rng, 1, 256)
        d_out = _log(rng, 1, 16384)
        group = rng.choice([g for g in (32, 64, 128, 256) if d_in % g == 0])
        p = min(64 * (d_out + d_in), d_out * d_in // 2) if rng.random() < 0.85 else 0
        return dict(op=op, act=act, T=_log(rng, 1, 64), d_out=d_out, d_in=d_in,
                    bits=rng.choice([4, 4, 4, 2, 3, 8]), group=group, p=p)
    kind = dict(op=op, act=act, dim=rng.choice([64, 128, 128, 256]),
                page=rng.choice([8, 16, 32, 64, 128]), bits=rng.choice([4, 4, 8]),
                rotate=rng.random() < 0.7)
    if op == "attn":
        length = _log(rng, 1, 65536)
        return dict(kind, B=_log(rng, 1, 64), kv_heads=rng.choice([1, 2, 3, 4, 8, 16]),
                    per_kv=rng.choice([1, 2, 3, 4, 5, 8, 12]), len=length,
                    shortest=rng.choice([0, 1, length // 2, length]))
    T = _log(rng, 1, 40000 if op == "read" else 8192)
    return dict(kind, T=T, heads=rng.choice([1, 2, 3, 5, 8, 16]),
                pages=T // kind["page"] + 1 + rng.randrange(64))


def draw(rng):
    """One case of the same ranges, no dearer than the dearest listed one."""
    most = max(_cost(c) for c in listed())
    while True:
        case = _drawn(rng)
        if _cost(case) <= most:
            return case


# ---------------------------------------------------------------- shapes and work
def _words(cols, bits):
    return -(-cols // (32 // bits))


def _lens(case):
    """The lengths of a ragged batch, evenly from the longest to the shortest."""
    B, hi, lo = case["B"], case["len"], case["shortest"]
    return [hi - (hi - lo) * i // max(B - 1, 1) for i in range(B)]


def _padding(case):
    """Rows of a batch of tokens that carry no token (slot -1)."""
    return case["T"] // 16


def work(case):
    e = 2 if case["act"] == "bf16" else 4
    if case["op"] == "decode":
        T, n, k, p = case["T"], case["d_out"], case["d_in"], case["p"]
        weights = n * (4 * _words(k, case["bits"]) + 8 * (k // case["group"]))
        adapter = 12 * p + 4 * (n + 1) if p else 0
        adds = T * k * math.log2(k & -k) if p else 0
        return {"bytes": e * T * (n + k) + weights + adapter,
                "flops": 2 * T * (n * k + p) + adds}
    d = case["dim"]
    row = 4 * _words(d, case["bits"]) + 8
    turn = math.log2(d) if case["rotate"] else 0
    if case["op"] == "attn":
        tokens, heads = sum(_lens(case)), case["kv_heads"]
        q_rows = case["B"] * heads * case["per_kv"]
        return {"bytes": 2 * tokens * heads * row + 2 * q_rows * d * e + 4 * case["B"]
                + 4 * sum(-(-n // case["page"]) for n in _lens(case)),
                "flops": 4 * tokens * heads * case["per_kv"] * d + 2 * q_rows * d * turn}
    T, live = case["T"], case["T"] - _padding(case)
    dense = 2 * e * case["heads"] * d
    stored = 2 * case["heads"] * row
    if case["op"] == "read":
        return {"bytes": live * stored + T * dense + 4 * T,
                "flops": 2 * live * case["heads"] * d * (2 + turn)}
    # written and read back: the dense rows in and out, the stored rows once
    return {"bytes": live * stored + (live + T) * dense + 4 * T,
            "flops": 2 * live * case["heads"] * d * (6 + 2 * turn)}


# ---------------------------------------------------------------- shared definitions
def _hadamard(n, dtype):
    """The Sylvester matrix: entry (i, j) is -1 to the number of bits that i and j share."""
    i = torch.arange(n, device=DEV)
    x = i[:, None] & i[None, :]
    x = x ^ (x >> 8)
    x = x ^ (x >> 4)
    x = x ^ (x >> 2)
    x = x ^ (x >> 1)
    return (1 - 2 * (x & 1)).to(dtype)


def _transform(x, n):
    """x H over the last dimension's blocks of n = 2^k, as the two factors of a Kronecker product."""
    lo = 1 << (n.bit_length() - 1) // 2
    y = x.reshape(-1, n // lo, lo)
    y = torch.matmul(y, _hadamard(lo, x.dtype))
    y = torch.matmul(_hadamard(n // lo, x.dtype), y)
    return y.reshape(x.shape)


def _unpack(words, bits, cols):
    """Codes of packed int32 words, along the last dimension."""
    cpw = 32 // bits
    at = torch.arange(cpw, device=words.device, dtype=torch.int32) * bits
    q = (words[..., None] >> at) & ((1 << bits) - 1)
    return q.reshape(*words.shape[:-1], words.shape[-1] * cpw)[..., :cols]


def _pack(q, bits):
    cpw = 32 // bits
    cols = q.shape[-1]
    nw = _words(cols, bits)
    q = torch.nn.functional.pad(q.to(torch.int64), (0, nw * cpw - cols))
    at = torch.arange(cpw, device=q.device) * bits
    w = (q.reshape(*q.shape[:-1], nw, cpw) << at).sum(-1)
    return torch.where(w >= 1 << 31, w - (1 << 32), w).to(torch.int32)


def _quantize(v, bits):
    """Codes, step and zero of each row of v (fp32): the row's range, zero included, in 2^bits - 1
    steps, halves rounded up. The step is held in fp32; which code a value gets is decided for that
    step, in 64 bits."""
    qmax = 2 ** bits - 1
    lo = v.amin(-1, keepdim=True).clamp(max=0.0)
    hi = v.amax(-1, keepdim=True).clamp(min=0.0)
    step = ((hi - lo).double() / qmax).float()
    flat = step < torch.finfo(torch.float32).tiny
    step = torch.where(flat, torch.zeros_like(step), step)
    by = torch.where(flat, torch.ones_like(step), step).double()
    zero = torch.where(flat, torch.zeros_like(by), torch.floor(-lo.double() / by + 0.5))
    q = torch.floor(v.double() / by + 0.5) + zero
    q = torch.where(flat, torch.zeros_like(q), q.clamp(0, qmax))
    return q.to(torch.int32), step[..., 0], zero[..., 0].float()


# ---------------------------------------------------------------- inputs
def _gen(seed):
    return torch.Generator(device=DEV).manual_seed(int(seed))


def _normal(g, *shape):
    return torch.randn(*shape, generator=g, device=DEV)


def _budgets(g, d_out, d_in, p):
    """Nonzeros of each row: shares of p that differ from row to row, as an allocation by the
    rows' quantization error gives them."""
    share = torch.exp(0.3 * _normal(g, d_out).double())
    n = torch.floor(p * share / share.sum()).to(torch.int64).clamp(max=d_in)
    left = p - int(n.sum())
    while left > 0:  # what rounding and full rows left over, one each
        room = torch.nonzero(n < d_in)[:left, 0]
        n[room] += 1
        left -= room.numel()
    return n


def _positions(g, n, d_in):
    """Distinct ascending columns for rows of n nonzeros: one in each of n even parts of the row."""
    p = int(n.sum())
    row = torch.repeat_interleave(torch.arange(n.numel(), device=DEV), n)
    ptr = torch.zeros(n.numel() + 1, dtype=torch.int64, device=DEV)
    ptr[1:] = torch.cumsum(n, 0)
    k = torch.arange(p, device=DEV) - ptr[row]
    parts = n[row]
    lo = -(-(k * d_in) // parts)
    hi = -(-((k + 1) * d_in) // parts)
    u = torch.rand(p, generator=g, device=DEV, dtype=torch.float64)
    col = lo + torch.floor(u * (hi - lo)).to(torch.int64).clamp(max=d_in - 1)
    col = torch.minimum(col, hi - 1)
    return ptr.to(torch.int32), torch.stack([row, col], 1).to(torch.int32).contiguous()


def _prepare_decode(case, g):
    T, n, k, bits, group, p = (case[f] for f in ("T", "d_out", "d_in", "bits", "group", "p"))
    w = 0.02 * _normal(g, n, k)
    w = torch.where(torch.rand(n, k, generator=g, device=DEV) < 0.001, 20 * w, w)
    w = w.reshape(n * (k // group), group)
    q, step, zero = _quantize(w, bits)
    state = dict(x=_normal(g, T, k).to(DTYPES[case["act"]]), alpha=0.75, bits=bits, group=group,
                 codes=_pack(q.reshape(n, k), bits).contiguous(),
                 scales=step.reshape(n, k // group).contiguous(),
                 zeros=zero.reshape(n, k // group).contiguous())
    ptr, E = _positions(g, _budgets(g, n, k, p), k)
    state.update(row_ptr=ptr, E=E, c=0.5 * _normal(g, p))
    return state


def _activations(g, rows, dim, act):
    """Keys or values: normal, with a few channels that stand out."""
    channel = torch.exp(0.3 * _normal(g, dim))
    channel[torch.randint(dim, (2,), generator=g, device=DEV)] *= 6
    return (_normal(g, rows, dim) * channel).to(act)


def _pool(g, pages, heads, page, dim, bits, rotate):
    """A cache filled with earlier tokens: codes [2][pages][heads][page][words], scales and zeros
    [2][pages][heads][page]; keys first, then values."""
    def part():
        v = _activations(g, pages * heads * page, dim, torch.bfloat16)
        v = (_transform(v.double(), dim) / dim).float() if rotate else v.float()
        q, step, zero = _quantize(v, bits)
        at = (pages, heads, page)
        return _pack(q, bits).reshape(*at, -1), step.reshape(at), zero.reshape(at)
    return [torch.stack(t).contiguous() for t in zip(part(), part())]


def _slots(g, case, contiguous):
    """A slot for each token, distinct; the batch's padding at the end has none. Read back are
    runs of tokens in page order, written are new tokens anywhere."""
    T, page, pages = case["T"], case["page"], case["pages"]
    if contiguous:
        order = torch.randperm(pages, generator=g, device=DEV)
        at = (order[:, None] * page + torch.arange(page, device=DEV)).reshape(-1)[:T].clone()
    else:
        at = torch.randperm(pages * page, generator=g, device=DEV)[:T].clone()
    at[T - _padding(case):] = -1
    return at.to(torch.int32)


def prepare(case, seed):
    g = _gen(seed)
    if case["op"] == "decode":
        return dict(_prepare_decode(case, g), op="decode")
    act, dim, bits = DTYPES[case["act"]], case["dim"], case["bits"]
    state = dict(op=case["op"], act=act, dim=dim, bits=bits, rotate=case["rotate"])
    if case["op"] == "attn":
        B, heads, page = case["B"], case["kv_heads"], case["page"]
        lens = torch.tensor(_lens(case), device=DEV)[torch.randperm(B, generator=g, device=DEV)]
        width = max(1, -(-case["len"] // page))
        used = (lens + page - 1) // page
        pages = max(1, sum(-(-n // page) for n in _lens(case)))
        first = torch.cumsum(used, 0) - used
        i = torch.arange(width, device=DEV)
        order = torch.randperm(pages, generator=g, device=DEV)
        table = order[(first[:, None] + i).clamp(max=pages - 1)]
        table = torch.where(i < used[:, None], table, torch.zeros_like(table))
        codes, scales, zeros = _pool(g, pages, heads, page, dim, bits, case["rotate"])
        q = _normal(g, B, heads * case["per_kv"], dim).to(act)
        return dict(state, q=q, codes=codes, scales=scales, zeros=zeros,
                    table=table.to(torch.int32).contiguous(), lens=lens.to(torch.int32))
    codes, scales, zeros = _pool(g, case["pages"], case["heads"], case["page"], dim, bits,
                                 case["rotate"])
    state.update(codes=codes, scales=scales, zeros=zeros,
                 slots=_slots(g, case, case["op"] == "read"))
    if case["op"] == "write":
        rows = case["T"] * case["heads"]
        k = _activations(g, rows, dim, act)
        v = _activations(g, rows, dim, act)
        state.update(k=k.reshape(case["T"], case["heads"], dim),
                     v=v.reshape(case["T"], case["heads"], dim))
    return state


# ---------------------------------------------------------------- plain forms
def _plain_decode(s):
    x = s["x"].float()
    n, k = s["codes"].shape[0], x.shape[1]
    q = _unpack(s["codes"], s["bits"], k).float().reshape(n, -1, s["group"])
    w = ((q - s["zeros"][..., None]) * s["scales"][..., None]).reshape(n, k)
    y = torch.matmul(x, w.t())
    if s["c"].numel():
        b = k & -k
        z = _transform(x.reshape(-1, b), b).reshape(x.shape) / b
        F = torch.zeros(n, k, device=x.device)
        F[s["E"][:, 0].long(), s["E"][:, 1].long()] = s["c"]
        y = y + s["alpha"] * torch.matmul(z, F.t())
    return y.to(s["x"].dtype)


def _plain_values(codes, scales, zeros, s):
    """Keys or values of gathered rows, in fp32."""
    v = (_unpack(codes, s["bits"], s["dim"]).float() - zeros[..., None]) * scales[..., None]
    return _transform(v, s["dim"]) if s["rotate"] else v


def _plain_write(s):
    keep = s["slots"] >= 0
    slots = s["slots"][keep].long()
    page = s["codes"].shape[3]
    x = torch.stack([s["k"][keep], s["v"][keep]])
    v = (_transform(x.double(), s["dim"]) / s["dim"]).float() if s["rotate"] else x.float()
    q, step, zero = _quantize(v, s["bits"])
    at = (slice(None), slots // page, slice(None), slots % page)
    # indexing by (page, row) puts the tokens first: [T][2][heads][...]
    s["codes"][at] = _pack(q, s["bits"]).transpose(0, 1).contiguous()
    s["scales"][at] = step.transpose(0, 1).contiguous()
    s["zeros"][at] = zero.transpose(0, 1).contiguous()


def _plain_read(s):
    keep = (s["slots"] >= 0)[:, None, None]
    slots = s["slots"].long().clamp(min=0)
    page = s["codes"].shape[3]
    at = (slice(None), slots // page, slice(None), slots % page)
    v = _plain_values(s["codes"][at], s["scales"][at], s["zeros"][at], s)
    v = torch.where(keep[:, None], v, torch.zeros_like(v)).to(s["act"])
    return [v[:, 0].contiguous(), v[:, 1].contiguous()]


def _plain_attn(s):
    q, table, lens = s["q"].float(), s["table"].long(), s["lens"].long()
    B, dim = q.shape[0], s["dim"]
    heads, page = s["codes"].shape[2], s["codes"].shape[3]
    L = table.shape[1] * page

    def part(i):  # [B][heads][L][dim]
        rows = [t[i][table].transpose(1, 2).reshape(B, heads, L, *t.shape[4:])
                for t in (s["codes"], s["scales"], s["zeros"])]
        return _plain_values(*rows, s)

    live = (torch.arange(L, device=q.device) < lens[:, None])[:, None, None]
    q = q.reshape(B, heads, -1, dim)
    a = torch.matmul(q, part(0).transpose(2, 3).contiguous()) / math.sqrt(dim)
    a = torch.where(live, a, torch.full_like(a, -torch.inf))
    top = a.amax(-1, keepdim=True)
    e = torch.exp(a - torch.where(torch.isfinite(top), top, torch.zeros_like(top)))
    total = e.sum(-1, keepdim=True)
    o = torch.matmul(e, part(1)) / torch.where(total > 0, total, torch.ones_like(total))
    return o.reshape(B, -1, dim).to(s["act"])


def run(state):
    s = state
    if own:
        import quantization_aware_sparse_amd as lib
        if s["op"] == "decode":
            return lib.qwha_layer_decode(s["x"], s["codes"], s["scales"], s["zeros"], s["bits"],
                                         s["group"], s["row_ptr"], s["E"], s["c"], s["alpha"])
        cache = (s["codes"], s["scales"], s["zeros"])
        if s["op"] == "attn":
            return lib.qwha_cache_attn(s["q"], *cache, s["table"], s["lens"], s["bits"],
                                       rotate=s["rotate"])
        if s["op"] == "write":
            lib.qwha_cache_write(s["k"], s["v"], s["slots"], *cache, s["bits"], rotate=s["rotate"])
        k, v = lib.qwha_cache_read(*cache, s["slots"], s["bits"], s["dim"], rotate=s["rotate"],
                                   out_dtype=s["act"])
        return [k, v, s["scales"], s["zeros"]] if s["op"] == "write" else [k, v]
    if s["op"] == "decode":
        return _plain_decode(s)
    if s["op"] == "attn":
        return _plain_attn(s)
    if s["op"] == "write":
        _plain_write(s)
        return [*_plain_read(s), s["scales"], s["zeros"]]
    return _plain_read(s)


# ---------------------------------------------------------------- 64 bits
def _sylvester(n):
    """H of order n by doubling: [[H, H], [H, -H]]."""
    h = torch.ones(1, 1, dtype=torch.float64, device=DEV)
    while h.shape[0] < n:
        h = torch.cat([torch.cat([h, h], 1), torch.cat([h, -h], 1)], 0)
    return h


def _digits(words, bits, cols):
    """Codes of packed words as float64: digit j % cpw, in base 2^bits, of word j / cpw."""
    cpw = 32 // bits
    j = torch.arange(cols, device=DEV)
    w = words.to(torch.int64)
    w = torch.where(w < 0, w + (1 << 32), w)
    out = torch.empty(*words.shape[:-1], cols, dtype=torch.float64, device=DEV)
    for i in range(cpw):
        here = j[i::cpw]
        out[..., here] = ((w[..., here // cpw] // (1 << (i * bits))) % (1 << bits)).double()
    return out


def _exact_decode(s):
    # the dense weights W_Q + alpha F H / b in 64 bits, and one product
    n, k = s["codes"].shape[0], s["x"].shape[1]
    b = k & -k
    w = torch.zeros(n, k, dtype=torch.float64, device=DEV)
    w.view(-1)[s["E"][:, 0].long() * k + s["E"][:, 1].long()] = s["c"].double()
    h = _sylvester(b) * (s["alpha"] / b)
    for j in range(0, k, b):
        w[:, j:j + b] = torch.matmul(w[:, j:j + b], h)
    del h
    group = torch.arange(k, device=DEV) // s["group"]
    w += ((_digits(s["codes"], s["bits"], k) - s["zeros"].double()[:, group])
          * s["scales"].double()[:, group])
    return torch.matmul(s["x"].double(), w.t())


def _exact_rows(s, part, page_of, row_of):
    """Stored tokens [tokens][heads][dim] in 64 bits."""
    words, step, zero = (t[part][page_of, :, row_of] for t in (s["codes"], s["scales"], s["zeros"]))
    v = (_digits(words, s["bits"], s["dim"]) - zero.double()[..., None]) * step.double()[..., None]
    return torch.matmul(v, _sylvester(s["dim"])) if s["rotate"] else v


def _exact_write(s):
    """What the cache holds afterwards. The stored row is fp32(x H / dim), its step is an fp32
    number by definition; the codes follow from both exactly."""
    scales, zeros, back = s["scales"].double(), s["zeros"].double(), []
    live = torch.nonzero(s["slots"] >= 0)[:, 0]
    slots = s["slots"][live].long()
    page = s["codes"].shape[3]
    qmax = float(2 ** s["bits"] - 1)
    for part, x in enumerate((s["k"], s["v"])):
        v = x[live].double()
        if s["rotate"]:
            v = torch.matmul(v, _sylvester(s["dim"])) / s["dim"]
        v = v.float().double()
        zero_in = torch.zeros_like(v[..., :1])
        both = torch.cat([v, zero_in], -1)
        lo, hi = both.min(-1).values, both.max(-1).values
        step = ((hi - lo).float().double() / qmax).float().double()
        step = torch.where(step < 2.0 ** -126, torch.zeros_like(step), step)
        by = torch.where(step > 0, step, torch.ones_like(step))
        zero = torch.where(step > 0, torch.floor(0.5 - lo / by), torch.zeros_like(step))
        code = torch.floor(0.5 + v / by[..., None]) + zero[..., None]
        code = torch.minimum(torch.maximum(code, torch.zeros_like(code)),
                             torch.full_like(code, qmax))
        scales[part][slots // page, :, slots % page] = step
        zeros[part][slots // page, :, slots % page] = zero
        out = torch.zeros(x.shape, dtype=torch.float64, device=DEV)
        v = (code - zero[..., None]) * step[..., None]
        out[live] = torch.matmul(v, _sylvester(s["dim"])) if s["rotate"] else v
        back.append(out)
    return [*back, scales, zeros]


def _exact_read(s):
    live = torch.nonzero(s["slots"] >= 0)[:, 0]
    slots = s["slots"][live].long()
    page = s["codes"].shape[3]
    back = []
    for part in range(2):
        out = torch.zeros(s["slots"].numel(), s["codes"].shape[2], s["dim"], dtype=torch.float64,
                          device=DEV)
        out[live] = _exact_rows(s, part, slots // page, slots % page)
        back.append(out)
    return back


def _exact_attn(s):
    # sequence by sequence, over its own tokens alone
    page = s["codes"].shape[3]
    heads = s["codes"].shape[2]
    out = torch.zeros(s["q"].shape, dtype=torch.float64, device=DEV)
    for i, n in enumerate(s["lens"].tolist()):
        if n == 0:
            continue
        t = torch.arange(n, device=DEV)
        page_of = s["table"][i].long()[t // page]
        k, v = (_exact_rows(s, part, page_of, t % page) for part in range(2))
        for h in range(heads):
            per = s["q"].shape[1] // heads
            rows = slice(h * per, (h + 1) * per)
            a = torch.matmul(s["q"][i, rows].double(), k[:, h].t()) * s["dim"] ** -0.5
            out[i, rows] = torch.matmul(torch.softmax(a, -1), v[:, h])
    return out


def exact(case, seed):
    s = prepare(case, seed)
    return {"decode": _exact_decode, "write": _exact_write, "read": _exact_read,
            "attn": _exact_attn}[case["op"]](s)
