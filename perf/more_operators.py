"""The cache and adapter operators of decoding: cases, inputs, plain forms and work.

  write   new keys and values into a paged cache of 8-bit codes (E4M3 or E5M2), one E8M0 scale per
          32 tokens and head; a block that grows takes a larger scale and rounds what it holds again
  read    tokens of the cache back, in bf16 or fp32
  attn    causal attention of a sequence's newest tokens over its cache
  lora    each token's own low-rank adapter beside a shared projection: base + s B (A x)

The cache: key codes [pages][heads][page][dim], value codes [pages][heads][page / 32][dim][32] (the 32
tokens of a block next to one another), scales [pages][heads][page / 32]; pages [sequences][..] is
the page table, lengths [sequences] counts a sequence's tokens, the new ones among them, and rows
offsets[b] .. offsets[b + 1] of the tokens are the newest ones of sequence b.

Sizes are the widths and heads of the 8B and 70B workloads (hidden 4096 and 8192, MLP 14336, heads of
128, key projections of 8 heads), their token counts, single tokens, and ragged ones.
"""
import math
import random

import torch

own = False

BF16, F32 = torch.bfloat16, torch.float32
DTYPES = {"bf16": BF16, "f32": F32}
F8 = {"e4m3": torch.float8_e4m3fn, "e5m2": torch.float8_e5m2}
E8 = torch.float8_e8m0fnu
LARGEST = {"e4m3": 448.0, "e5m2": 57344.0}
EMAX = {"e4m3": 8, "e5m2": 15}
BLOCK = 32


def _cache(name, op, seqs, length, new, heads, dim, page, dtype="bf16", fmt="e4m3", **more):
    """length and new: (least, most) tokens of a sequence and of its newest ones."""
    return {"name": name, "op": op, "seqs": seqs, "len_lo": length[0], "len_hi": length[1],
            "new_lo": new[0], "new_hi": new[1], "heads": heads, "dim": dim, "page": page,
            "dtype": dtype, "fmt": fmt, "plan": 7 * seqs + length[1], **more}


def _lora(name, T, N, K, rank, adapters, dtype="bf16", run=1, base="f32"):
    """run: how many tokens in a row have the same adapter."""
    return {"name": name, "op": "lora", "T": T, "N": N, "K": K, "rank": rank,
            "adapters": adapters, "dtype": dtype, "run": run, "base": base, "plan": T + N}


def listed():
    return [
        # a decoding step of 64 sequences of the 70B model: one new token each
        _cache("write_tokens_70b", "write", 64, (1000, 9000), (1, 1), 8, 128, 64),
        # prompts of four requests that arrive together, 8192 tokens in all
        _cache("write_prompts_8b", "write", 4, (2048, 2048), (2048, 2048), 8, 128, 64),
        # pieces of prompts behind what is cached, fp32, wide range, the truncation-free scale
        _cache("write_ragged_f32", "write", 5, (300, 3000), (1, 290), 3, 64, 96, dtype="f32",
               fmt="e5m2", ceil=True),
        # a shared prompt back in bf16, for a path that wants it whole
        _cache("read_prompts_8b", "read", 8, (500, 4000), (500, 4000), 8, 128, 64),
        # the last tokens of three sequences, fp32, wide heads
        _cache("read_tail_f32", "read", 3, (100, 5000), (20, 70), 2, 256, 32, dtype="f32",
               fmt="e5m2"),
        # one request of the 8B model: 32 query heads over 8 of the cache, latency
        _cache("attn_token_8b", "attn", 1, (2000, 2100), (1, 1), 8, 128, 64, group=4),
        # 64 requests of the 70B model (64 query heads over 8), lengths far apart
        _cache("attn_batch_70b", "attn", 64, (500, 16000), (1, 1), 8, 128, 64, group=8),
        # one request with a very long context
        _cache("attn_long_70b", "attn", 1, (262000, 262100), (1, 1), 8, 128, 128, group=8),
        # a few drafted tokens of each request are checked at once, fp32, ragged
        _cache("attn_draft_f32", "attn", 12, (40, 6000), (1, 9), 4, 64, 96, dtype="f32",
               fmt="e5m2", group=3),
        # one request's token beside the 8B up projection, eight adapters loaded
        _lora("lora_token_8b", 1, 14336, 4096, 16, 8),
        # 64 requests with 32 adapters beside a square 70B projection
        _lora("lora_batch_70b", 64, 8192, 8192, 16, 32),
        # prompts of several requests through the 8B up projection
        _lora("lora_prompts_8b", 2048, 14336, 4096, 64, 4, run=300),
    ]


def _log_int(rng, lo, hi):
    return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["write", "read", "attn", "lora"])
    dtype = rng.choice(["bf16", "bf16", "f32"])
    if op == "lora":
        T = _log_int(rng, 1, 2048)
        n = _log_int(rng, 17, 14336)
        return {"op": op, "T": T, "N": n, "K": 32 * _log_int(rng, 4, 256),
                "rank": 8 * _log_int(rng, 1, 8), "adapters": _log_int(rng, 1, 64), "dtype": dtype,
                "run": rng.choice([1, 1, 7, 300]), "base": rng.choice(["f32", "same", "none"]),
                "plan": rng.randrange(1 << 20)}
    dim = rng.choice([64, 128, 128, 192, 256])
    heads = rng.choice([1, 2, 3, 8])
    seqs = _log_int(rng, 1, 64)
    # tokens x heads x dim of all sequences
    most = (8192 * 1024 if op != "attn" else 1 << 29) // (heads * dim * seqs)
    hi = _log_int(rng, 1, max(1, min(most, 65536)))
    lo = _log_int(rng, 1, hi)
    if op == "attn":
        new = rng.choice([(1, 1), (1, 1), (1, 12)])
    else:
        new = rng.choice([(1, 1), (1, hi), (hi, hi)])
    case = {"op": op, "seqs": seqs, "len_lo": lo, "len_hi": hi, "new_lo": new[0],
            "new_hi": new[1], "heads": heads, "dim": dim, "page": rng.choice([32, 64, 96, 128]),
            "dtype": dtype, "fmt": rng.choice(["e4m3", "e4m3", "e5m2"]),
            "plan": rng.randrange(1 << 20)}
    if op == "write":
        case["ceil"] = rng.random() < 0.5
    if op == "attn":
        case["group"] = rng.choice([1, 3, 4, 8])
    return case


def _plan(case):
    """Lengths and newest tokens of the sequences, or the adapter of each token (-1: none); they
    are the case's, whatever the seed of the inputs."""
    rng = random.Random(case["plan"])
    if case["op"] == "lora":
        index, t = [], 0
        while t < case["T"]:
            a = rng.randrange(case["adapters"]) if rng.random() < 0.95 else -1
            for _ in range(min(rng.randint(1, 2 * case["run"] - 1), case["T"] - t)):
                index.append(a)
                t += 1
        return index
    lengths = [rng.randint(case["len_lo"], case["len_hi"]) for _ in range(case["seqs"])]
    new = [min(n, rng.randint(case["new_lo"], case["new_hi"])) for n in lengths]
    return lengths, new


def work(case):
    e = 2 if case["dtype"] == "bf16" else 4
    if case["op"] == "lora":
        index = _plan(case)
        T, N, K, r = case["T"], case["N"], case["K"], case["rank"]
        with_one = sum(a >= 0 for a in index)
        used = len({a for a in index if a >= 0})
        b = with_one * K * e + used * r * (N + K) * e + T * N * e + 4 * T + 4 * used
        b += T * N * {"f32": 4, "same": e, "none": 0}[case["base"]]
        return {"bytes": b, "flops": 2 * with_one * r * (N + K) + 2 * T * N}
    lengths, new = _plan(case)
    H, D = case["heads"], case["dim"]
    tokens = sum(new)
    table = sum(-(-n // case["page"]) for n in lengths) * 4 + 12 * case["seqs"]
    if case["op"] == "attn":
        held = sum(lengths)
        pairs = sum(n * l - n * (n - 1) // 2 for l, n in zip(lengths, new))
        G = case["group"]
        return {"bytes": held * H * D * 2 + held * H // 16 + 2 * tokens * H * G * D * e + table,
                "flops": 4 * pairs * H * G * D}
    blocks = sum(-(-l // BLOCK) - (l - n) // BLOCK for l, n in zip(lengths, new))
    return {"bytes": 2 * tokens * H * D * (e + 1) + 2 * blocks * H + table,
            "flops": 4 * tokens * H * D}


# ------------------------------------------------------------------------------------------------
# inputs
# ------------------------------------------------------------------------------------------------
def _randn(gen, *shape):
    return torch.randn(shape, generator=gen, device="cuda", dtype=F32)


def _exponent(amax, fmt, ceil=False):
    """Biased scale exponent of a block's largest magnitude (fp32)."""
    bits = amax.view(torch.int32)
    e = (bits >> 23) - EMAX[fmt]
    if ceil:
        e = e + ((bits & 0x7FFFFF) > 0x600000).to(torch.int32)
    return e.clamp(min=0)


def _to_codes(v, e, fmt):
    """v in fp32, e its blocks' biased exponents, of a shape that broadcasts."""
    big = LARGEST[fmt]
    return torch.ldexp(v, 127 - e).clamp(-big, big).to(F8[fmt])


def _fill(gen, case, pages):
    """A cache full of tokens: channels of different size, tokens too."""
    H, D, P = case["heads"], case["dim"], case["page"]
    shape = (pages, H, P // BLOCK)
    st = {"kq": torch.empty((pages, H, P, D), dtype=torch.uint8, device="cuda"),
          "vq": torch.empty(shape + (D, BLOCK), dtype=torch.uint8, device="cuda"),
          "ks": torch.empty(shape, dtype=torch.uint8, device="cuda"),
          "vs": torch.empty(shape, dtype=torch.uint8, device="cuda")}
    gain = {"k": torch.exp(0.8 * _randn(gen, H, 1, 1, D)), "v": torch.exp(0.3 * _randn(gen, H, 1, 1, D))}
    gain["k"] = gain["k"] / gain["k"].square().mean().sqrt()
    step = max(1, (1 << 25) // (H * P * D))
    for p in range(0, pages, step):
        n = min(step, pages - p)
        for x in "kv":
            v = _randn(gen, n, H, P // BLOCK, BLOCK, D)
            v.mul_(torch.exp(0.3 * _randn(gen, n, H, P // BLOCK, BLOCK, 1))).mul_(gain[x])
            e = _exponent(v.abs().amax((3, 4)), case["fmt"])
            q = _to_codes(v, e[..., None, None], case["fmt"]).view(torch.uint8)
            st[x + "s"][p:p + n] = e.to(torch.uint8)
            if x == "k":
                st["kq"][p:p + n] = q.view(n, H, P, D)
            else:
                st["vq"][p:p + n] = q.transpose(3, 4)
    return st


def _tables(gen, case, lengths, new):
    """Pages in any order, a few of the cache's to spare, -1 behind a sequence's last one."""
    need = [-(-n // case["page"]) for n in lengths]
    total = sum(need) + 3
    order = torch.randperm(total, generator=gen, device="cuda").to(torch.int32)
    width = max(need) + 1
    starts = [sum(need[:b]) for b in range(len(need))]
    at = torch.arange(width, device="cuda")
    need_t = torch.tensor(need, device="cuda")[:, None]
    first = torch.tensor(starts, device="cuda")[:, None]
    pages = torch.where(at < need_t, order[(first + at).clamp(max=total - 1)],
                        torch.tensor(-1, dtype=torch.int32, device="cuda"))
    sums = [sum(new[:b]) for b in range(len(new) + 1)]
    return total, {"pages": pages.to(torch.int32).contiguous(),
                   "lengths": torch.tensor(lengths, dtype=torch.int32, device="cuda"),
                   "offsets": torch.tensor(sums, dtype=torch.int32, device="cuda")}


def prepare(case, seed):
    gen = torch.Generator(device="cuda")
    gen.manual_seed(int(seed) * 7919 + 23)
    dtype = DTYPES[case["dtype"]]
    st = {"case": case, "plan": _plan(case)}
    if case["op"] == "lora":
        T, N, K, r, E = (case[k] for k in ("T", "N", "K", "rank", "adapters"))
        st["x"] = _randn(gen, T, K)
        at = torch.randint(0, K, (max(1, K // 200),), generator=gen, device="cuda")
        st["x"][:, at] *= 20.0
        st["x"] = st["x"].to(dtype)
        st["a"] = (_randn(gen, E, r, K) * K ** -0.5).to(dtype)
        st["b"] = (_randn(gen, E, N, r) * 0.02).to(dtype)
        st["scaling"] = 0.5 + 1.5 * torch.rand(E, generator=gen, device="cuda")
        st["index"] = torch.tensor(st["plan"], dtype=torch.int32, device="cuda")
        st["base"] = None if case["base"] == "none" else \
            _randn(gen, T, N).to(F32 if case["base"] == "f32" else dtype)
        return st
    lengths, new = st["plan"]
    pages, tables = _tables(gen, case, lengths, new)
    st.update(tables)
    st.update(_fill(gen, case, pages))
    T, H, D = sum(new), case["heads"], case["dim"]
    if case["op"] == "write":
        # keys and values as a joint projection leaves them, tokens of different size: some make
        # their block's scale grow
        kv = _randn(gen, T, 2, H, D) * torch.exp(_randn(gen, T, 2, H, 1))
        kv = kv.to(dtype)
        st["k"], st["v"] = kv[:, 0], kv[:, 1]
    elif case["op"] == "attn":
        st["q"] = (2.0 * _randn(gen, T, H * case["group"], D)).to(dtype)
    return st


# ------------------------------------------------------------------------------------------------
# one pass
# ------------------------------------------------------------------------------------------------
def run(state):
    case = state["case"]
    if own:
        return _run_own(state, case)
    return {"write": _plain_write, "read": _plain_read, "attn": _plain_attn,
            "lora": _plain_lora}[case["op"]](state, case)


def _whole(st, case):
    """The updated cache: codes and scales as the values that they stand for."""
    f8 = F8[case["fmt"]]
    return {"kq": st["kq"].view(f8), "vq": st["vq"].view(f8), "ks": st["ks"].view(E8),
            "vs": st["vs"].view(E8)}


def _run_own(st, case):
    import mxfp4_block_scaled_hadamard32_amd as mx
    if case["op"] == "lora":
        return mx.mx_lora(st["x"], st["a"], st["b"], st["index"], base=st["base"],
                          scaling=st["scaling"], out_dtype=st["x"].dtype)
    fmt = mx.MX_E4M3 if case["fmt"] == "e4m3" else mx.MX_E5M2
    cache = (st["kq"], st["ks"], st["vq"], st["vs"], st["pages"], st["lengths"])
    # without offsets every sequence has one new token
    offsets = None if case["new_hi"] == 1 else st["offsets"]
    if case["op"] == "write":
        rule = mx.MX_SCALE_CEIL if case.get("ceil") else mx.MX_SCALE_FLOOR
        mx.mx_cache_write(st["k"], st["v"], *cache, offsets=offsets, fmt=fmt, scale_rule=rule)
        return _whole(st, case)
    if case["op"] == "read":
        return mx.mx_cache_read(*cache, offsets=offsets, rows=sum(st["plan"][1]), fmt=fmt,
                                out_dtype=DTYPES[case["dtype"]])
    return mx.mx_cache_attention(st["q"], *cache, offsets=offsets, fmt=fmt)


def _span(st, b, case):
    """Block numbers (first, end) of a sequence's newest tokens and the first one's position."""
    length, n = st["plan"][0][b], st["plan"][1][b]
    return (length - n) // BLOCK, -(-length // BLOCK), length - n


def _where(st, case):
    """Page and block within it of every block that holds a newest token; the row of the tokens
    that its first slot would have; how many slots at its start are older, how many are filled."""
    P = case["page"] // BLOCK
    rows, row = [], 0
    for b in range(case["seqs"]):
        first, end, start = _span(st, b, case)
        length, n = st["plan"][0][b], st["plan"][1][b]
        for i in range(first, end):
            rows.append((b, i, row + i * BLOCK - start, max(0, start - i * BLOCK),
                         min(BLOCK, length - i * BLOCK)))
        row += n
    t = torch.tensor(rows, device="cuda")
    page = st["pages"][t[:, 0], t[:, 1] // P].long()
    return page, t[:, 1] % P, t[:, 2], t[:, 3], t[:, 4]


def _plain_write(st, case):
    H, D, fmt = case["heads"], case["dim"], case["fmt"]
    f8 = F8[fmt]
    page, at, row, old, filled = _where(st, case)
    slot = torch.arange(BLOCK, device="cuda")
    fresh = ((slot >= old[:, None]) & (slot < filled[:, None]))[:, None, :, None]
    kept = (slot < old[:, None])[:, None, :, None]
    source = (row[:, None] + slot).clamp(0, st["k"].shape[0] - 1)
    for x in "kv":
        new = st[x][source].float().transpose(1, 2)  # [blocks][H][32][D]
        new = torch.where(fresh, new, 0.0)
        e = _exponent(new.abs().amax((2, 3)), fmt, case.get("ceil", False))
        s = st[x + "s"][page, :, at].to(torch.int32)
        e = torch.where(old[:, None] > 0, torch.maximum(e, s), e)
        if x == "k":
            view = st["kq"].view(-1, H, case["page"] // BLOCK, BLOCK, D)
            held = view[page, :, at]
        else:
            view = st["vq"]
            held = view[page, :, at].transpose(2, 3)
        # what is there already, rounded again where the scale has grown
        again = _to_codes(held.contiguous().view(f8).float(), (127 + e - s)[:, :, None, None], fmt)
        q = torch.where(fresh, _to_codes(new, e[:, :, None, None], fmt).view(torch.uint8),
                        torch.where(kept, again.view(torch.uint8), held))
        view[page, :, at] = q if x == "k" else q.transpose(2, 3)
        st[x + "s"][page, :, at] = e.to(torch.uint8)
    return _whole(st, case)


def _decode(st, x, page, at, case):
    """Blocks of the cache in fp32, [..][H][32][D]."""
    H, D = case["heads"], case["dim"]
    if x == "k":
        q = st["kq"].view(-1, H, case["page"] // BLOCK, BLOCK, D)[page, :, at]
    else:
        q = st["vq"][page, :, at].transpose(-1, -2).contiguous()
    e = st[x + "s"][page, :, at].to(torch.int32)
    return torch.ldexp(q.view(F8[case["fmt"]]).float(), (e - 127)[..., None, None])


def _plain_read(st, case):
    page, at, row, old, filled = _where(st, case)
    slot = torch.arange(BLOCK, device="cuda")
    fresh = (slot >= old[:, None]) & (slot < filled[:, None])
    target = (row[:, None] + slot)[fresh]
    out = []
    for x in "kv":
        v = _decode(st, x, page, at, case).transpose(1, 2)[fresh]  # [tokens][H][D]
        o = torch.empty_like(v)
        o[target] = v
        out.append(o.to(DTYPES[case["dtype"]]))
    return tuple(out)


def _plain_attn(st, case):
    H, D, G, P = case["heads"], case["dim"], case["group"], case["page"] // BLOCK
    out, row = torch.empty_like(st["q"]), 0
    for b in range(case["seqs"]):
        length, n = st["plan"][0][b], st["plan"][1][b]
        i = torch.arange(-(-length // BLOCK), device="cuda")
        page = st["pages"][b, i // P].long()
        k, v = (_decode(st, x, page, i % P, case).transpose(0, 1).reshape(H, -1, D)[:, :length]
                for x in "kv")
        q = st["q"][row:row + n].float().view(n, H, G, D).transpose(0, 1).reshape(H, n * G, D)
        s = torch.matmul(q, k.transpose(1, 2).contiguous()) * D ** -0.5
        if n > 1:
            pos = torch.arange(length, device="cuda")
            last = length - n + torch.arange(n, device="cuda").repeat_interleave(G)
            s = s.masked_fill(pos > last[:, None], -math.inf)
        p = torch.exp(s - s.amax(2, keepdim=True))
        o = torch.matmul(p, v.contiguous()) / p.sum(2, keepdim=True)
        out[row:row + n] = o.view(H, n, G, D).transpose(0, 1).reshape(n, H * G, D).to(out.dtype)
        row += n
    return out


def _plain_lora(st, case):
    x, index = st["x"].float(), st["index"]
    y = torch.zeros((case["T"], case["N"]), device="cuda") if st["base"] is None \
        else st["base"].float()
    used = sorted({a for a in st["plan"] if a >= 0})
    for a in used:
        rows = torch.nonzero(index == a)[:, 0]
        h = torch.matmul(x[rows], st["a"][a].float().t().contiguous()) * st["scaling"][a]
        y = y.index_add(0, rows, torch.matmul(h, st["b"][a].float().t().contiguous()))
    return y.to(st["x"].dtype)


# ------------------------------------------------------------------------------------------------
# the definition in 64 bits
# ------------------------------------------------------------------------------------------------
def _round_f64(v, fmt):
    """v to the nearest value of the format, ties to even, saturated."""
    bits, least = (3, -6) if fmt == "e4m3" else (2, -14)
    big = LARGEST[fmt]
    v = v.clamp(-big, big)
    step = torch.exp2(((torch.frexp(v).exponent - 1).clamp_(min=least) - bits).double())
    return (torch.round(v / step) * step).clamp_(-big, big)


def _exact_write(st, case):
    fmt, D, P = case["fmt"], case["dim"], case["page"]
    res = {"kq": st["kq"].view(F8[fmt]).to(F32).double(), "vq": st["vq"].view(F8[fmt]).to(F32).double(),
           "ks": torch.exp2(st["ks"].double() - 127), "vs": torch.exp2(st["vs"].double() - 127)}
    lengths, new = st["plan"]
    table = st["pages"].tolist()
    row = 0
    for b in range(case["seqs"]):
        start, pos = lengths[b] - new[b], lengths[b] - new[b]
        while pos < lengths[b]:  # one block after the other
            i, at = table[b][pos // P], pos % P // BLOCK
            lo = pos % BLOCK
            n = min(BLOCK - lo, lengths[b] - pos)
            r = row + pos - start
            for x in "kv":
                w = st[x][r:r + n].double().transpose(0, 1)  # [H][n][D]
                mant, ex = torch.frexp(w.abs().amax((1, 2)))
                e = ex.double() - 1 - EMAX[fmt]
                if case.get("ceil", False):
                    e = e + (mant > 0.875).double()
                scale = torch.exp2(e.clamp(min=-127.0))
                held = res["kq"][i, :, at * BLOCK:(at + 1) * BLOCK] if x == "k" else \
                    res["vq"][i, :, at].transpose(1, 2)
                if lo:
                    was = res[x + "s"][i, :, at]
                    scale = torch.maximum(scale, was)
                    held[:, :lo] = _round_f64(held[:, :lo] * (was / scale)[:, None, None], fmt)
                held[:, lo:lo + n] = _round_f64(w / scale[:, None, None], fmt)
                res[x + "s"][i, :, at] = scale
            pos += n
        row += new[b]
    return res


def _sequence_f64(st, case, b, x, first, count):
    """`count` tokens of a sequence from position `first` on, [count][H][D]."""
    P, D, H = case["page"], case["dim"], case["heads"]
    pos = first + torch.arange(count, device="cuda")
    page = st["pages"][b][pos // P].long()
    h = torch.arange(H, device="cuda")
    if x == "k":
        q = st["kq"][page[:, None], h, (pos % P)[:, None]]
    else:
        q = st["vq"].permute(0, 1, 2, 4, 3)[page[:, None], h, (pos % P // BLOCK)[:, None],
                                            (pos % BLOCK)[:, None]]
    e = st[x + "s"][page[:, None], h, (pos % P // BLOCK)[:, None]]
    return q.contiguous().view(F8[case["fmt"]]).to(F32).double() * torch.exp2(e.double() - 127)[:, :, None]


def exact(case, seed):
    st = prepare(case, seed)
    if case["op"] == "write":
        return _exact_write(st, case)
    if case["op"] == "lora":
        y = torch.zeros((case["T"], case["N"]), dtype=torch.float64, device="cuda")
        index = torch.tensor(st["plan"], device="cuda")
        for a in range(case["adapters"]):
            rows = (index == a).nonzero().flatten()
            if len(rows):
                h = st["x"][rows].double() @ st["a"][a].double().T
                y[rows] = h @ st["b"][a].double().T * st["scaling"][a].double()
        return y if st["base"] is None else y + st["base"].double()
    lengths, new = st["plan"]
    D = case["dim"]
    if case["op"] == "read":
        return tuple(torch.cat([_sequence_f64(st, case, b, x, l - n, n)
                                for b, (l, n) in enumerate(zip(lengths, new))]) for x in "kv")
    out, row, G = [], 0, case["group"]
    for b, (l, n) in enumerate(zip(lengths, new)):
        k, v = (_sequence_f64(st, case, b, x, 0, l) for x in "kv")
        heads = []
        for h in range(case["heads"]):
            q = st["q"][row:row + n, h * G:(h + 1) * G].double()
            rows = []
            for t in range(n):
                seen = l - n + t + 1
                w = torch.softmax(q[t] @ k[:seen, h].T / math.sqrt(D), 1)
                rows.append(w @ v[:seen, h])
            heads.append(torch.stack(rows))          # [n][G][D]
        out.append(torch.cat(heads, 1))
        row += n
    return torch.cat(out)
