"""What sliding-window attention over the paged cache costs, and the tables built on the GPU for it.

Four operators are measured:

* ``decode``  one new token a request over bf16 pages (``oxd_window_decode``);
* ``quant``   the same over a cache held in 4 bits (``oxd_quant_window_decode``);
* ``prefill`` causal prefill with a window (``oxd_window_prefill_plan``, ``oxd_paged_prefill_run``);
* ``tables``  block tables, token maps and slots from request lengths (``oxd_build_tables``).

A query at position p of its request sees the cached tokens j <= p with j > p - window (the
window) or j < sinks (the first tokens, which stay visible). Pages that no query of a call sees
are not held any more: the block tables list them as -1.

The 4-bit format: the 128 values of one (token, KV head) are four groups of 32, a group's scale
the f16 nearest to amax / 6, a value's code the e2m1 number (0, 0.5, 1, 1.5, 2, 3, 4, 6 and their
negatives) nearest to value / scale. Two codes a byte, the even column in the low half; codes
[pages, page_size, heads, 64] (NHD) or [pages, heads, page_size, 64] (HND), scales
[pages, heads, page_size, 4] f16.
"""
import math

import numpy as np
import torch

own = False

DEVICE = "cuda"
LEVELS = (0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0)


# ------------------------------------------------------------------ cases

def listed():
    return [
        # one request, a chat past its window: latency
        dict(name="decode_b1_w1024", kind="decode", batch=1, hq=32, hkv=8, ps=16, layout="NHD",
             lo=4096, hi=4096, window=1024, sinks=4),
        # a serving batch, short and long requests, a small window
        dict(name="decode_b64_w512", kind="decode", batch=64, hq=32, hkv=8, ps=16, layout="HND",
             lo=100, hi=8192, window=512, sinks=0),
        # long documents, one KV head for 32 query heads
        dict(name="decode_mqa32_b16_w8192", kind="decode", batch=16, hq=32, hkv=1, ps=64,
             layout="NHD", lo=32768, hi=32768, window=8192, sinks=64),
        # the largest batch of the decode benchmark
        dict(name="decode_gqa8_b256_w4096", kind="decode", batch=256, hq=64, hkv=8, ps=16,
             layout="NHD", lo=128, hi=16384, window=4096, sinks=4),
        # a few requests over a 4-bit cache: latency
        dict(name="quant_b8_w1024", kind="quant", batch=8, hq=32, hkv=8, ps=16, layout="NHD",
             lo=2048, hi=8192, window=1024, sinks=4),
        # the largest batch over a 4-bit cache
        dict(name="quant_gqa8_b256_w4096", kind="quant", batch=256, hq=64, hkv=8, ps=16,
             layout="NHD", lo=128, hi=16384, window=4096, sinks=4),
        # two short turns on two chats
        dict(name="prefill_turns_w512", kind="prefill", hq=32, hkv=8, ps=16, layout="NHD",
             q="32 64", kv="256 1024", window=512, sinks=4),
        # a chunk of a long document
        dict(name="prefill_chunk_w4096", kind="prefill", hq=32, hkv=8, ps=16, layout="HND",
             q="1000", kv="16384", window=4096, sinks=16),
        # prompts of a batch
        dict(name="prefill_prompts_w1024", kind="prefill", hq=32, hkv=8, ps=16, layout="NHD",
             q=" ".join(["2048"] * 8), kv="2048 4096 6144 8192 10240 12288 14336 16384", window=1024,
             sinks=4),
        # the tables of one decode step
        dict(name="tables_step_b64", kind="tables", batch=64, ps=16, lo=100, hi=8192, new=1,
             window=0, sinks=0),
        # the tables of prompts of odd lengths
        dict(name="tables_prompts_b8", kind="tables", batch=8, ps=16, lo=2047, hi=16384, new=2047,
             window=1024, sinks=4),
        # the tables of one decode step of the largest batch that a pool holds
        dict(name="tables_step_b1024", kind="tables", batch=1024, ps=16, lo=128, hi=16384, new=1,
             window=4096, sinks=4),
    ]


def _counts(text):
    """The numbers of a text, one a request."""
    return [int(x) for x in text.split()]


def _log_uniform(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    kind = rng.choice(["decode", "decode", "quant", "prefill", "prefill", "tables"])
    ps = rng.choice([8, 16, 32, 64])
    layout = rng.choice(["NHD", "HND"])
    hkv = rng.choice([1, 2, 3, 4, 8])
    group = rng.choice([1, 2, 4, 5, 8, 16, 32])
    window = _log_uniform(rng, 16, 8192)
    sinks = rng.choice([0, 1, 4, 16, 100])
    if kind in ("decode", "quant"):
        most = 8_000_000 if kind == "decode" else 7_000_000  # tokens x heads
        batch = _log_uniform(rng, 1, 256)
        window = min(window, max(16, most // (batch * hkv) - sinks))
        hi = _log_uniform(rng, 2, 32768)
        return dict(kind=kind, batch=batch, hq=group * hkv, hkv=hkv, ps=ps, layout=layout,
                    lo=rng.choice([1, max(1, hi // 4), hi]), hi=hi, window=window, sinks=sinks)
    if kind == "prefill":
        group = min(group, max(1, 64 // hkv))
        q, kv = [], []
        left = 16384 * 32 * 1024 // (group * hkv) // (window + sinks)  # query tokens
        for _ in range(rng.choice([1, 2, 3, 8])):
            n = min(_log_uniform(rng, 1, 4096), left)
            if n < 1:
                break
            left -= n
            q.append(n)
            kv.append(n + rng.choice([0, rng.randrange(0, 300), rng.randrange(0, 12000)]))
        return dict(kind=kind, hq=group * hkv, hkv=hkv, ps=ps, layout=layout,
                    q=" ".join(map(str, q)), kv=" ".join(map(str, kv)), window=window, sinks=sinks)
    batch = _log_uniform(rng, 1, 1024)
    hi = _log_uniform(rng, 2, min(32768, 1024 * 8192 // batch))
    new = rng.choice([1, _log_uniform(rng, 1, max(1, min(hi, 16384 // batch)))])
    return dict(kind=kind, batch=batch, ps=ps, lo=rng.choice([1, max(1, hi // 4), hi]), hi=hi,
                new=new, window=rng.choice([0, window]), sinks=sinks)


# ------------------------------------------------------------------ inputs

def _generator(seed):
    return torch.Generator(device=DEVICE).manual_seed(seed)


def _randn(shape, g):
    return torch.randn(shape, generator=g, device=DEVICE, dtype=torch.float32).to(torch.bfloat16)


def _device(a):
    return torch.as_tensor(a, device=DEVICE)


def _pool_shape(case, pages, width):
    ps, h = case["ps"], case["hkv"]
    return (pages, ps, h, width) if case["layout"] == "NHD" else (pages, h, ps, width)


def _dead_pages(case, pages, first_query):
    """Of a request's pages, those that no query from position first_query on sees."""
    j = np.arange(pages)
    return (j * case["ps"] >= case["sinks"]) & ((j + 1) * case["ps"] <= first_query + 1 - case["window"])


def _tables(case, lengths, first_query, rng):
    """CSR tables over a shuffled pool of the pages still held, a few more in the pool."""
    ps = case["ps"]
    pages = -(-lengths // ps)
    indptr = np.concatenate([[0], np.cumsum(pages)]).astype(np.int32)
    dead = np.concatenate([_dead_pages(case, n, f) for n, f in zip(pages, first_query)])
    pool = int((~dead).sum()) + 3
    indices = np.full(len(dead), -1, np.int32)
    indices[~dead] = rng.permutation(pool)[:pool - 3]
    return indptr, indices, (lengths - (pages - 1) * ps).astype(np.int32), pool


def _fill(shape, g, step=1 << 27):
    """Normal values in bf16, made in parts."""
    out = torch.empty(shape, dtype=torch.bfloat16, device=DEVICE)
    flat = out.view(-1)
    for i in range(0, flat.numel(), step):
        flat[i:i + step] = _randn((min(step, flat.numel() - i),), g)
    return out


def _packed(case, pages, g):
    """Normal values held in 4 bits: codes and scales."""
    codes = torch.empty(_pool_shape(case, pages, 64), dtype=torch.uint8, device=DEVICE)
    scales = torch.empty((pages, case["hkv"], case["ps"], 4), dtype=torch.float16, device=DEVICE)
    step = max(1, (1 << 26) // (case["ps"] * case["hkv"] * 128))
    for p in range(0, pages, step):
        n = min(step, pages - p)
        x = _randn(_pool_shape(case, n, 128), g).float().unflatten(-1, (4, 32))
        s = (x.abs().amax(-1) / 6.0).half()
        y = x / s.float().clamp(min=1e-7).unsqueeze(-1)
        a = y.abs()
        code = 8 * (y < 0).byte()
        for border in (0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0):
            code += (a > border).byte()
        code = code.flatten(-2)
        codes[p:p + n] = code[..., 0::2] + 16 * code[..., 1::2]
        scales[p:p + n] = s.transpose(1, 2) if case["layout"] == "NHD" else s
    return codes, scales


def _prepare_decode(case, seed):
    rng, g = np.random.default_rng(seed), _generator(seed)
    lengths = rng.integers(case["lo"], case["hi"] + 1, case["batch"])
    indptr, indices, last, pool = _tables(case, lengths, lengths - 1, rng)
    s = dict(case=case, lengths=_device(lengths), indptr=_device(indptr), indices=_device(indices),
             last=_device(last), scale=1.0 / math.sqrt(128),
             q=_randn((case["batch"], case["hq"], 128), g))
    if case["kind"] == "quant":
        s["k"], s["ks"] = _packed(case, pool, g)
        s["v"], s["vs"] = _packed(case, pool, g)
    else:
        s["k"] = _fill(_pool_shape(case, pool, 128), g)
        s["v"] = _fill(_pool_shape(case, pool, 128), g)
    s["out"] = torch.empty_like(s["q"])
    s["lse"] = torch.empty((case["batch"], case["hq"]), device=DEVICE)
    if own:
        import paged_kv_decode_attn_gb300 as oxd

        s["desc"] = oxd.make_window_decode_desc(
            case["batch"], case["hq"], case["hkv"], case["ps"], case["layout"], pool,
            len(indices), case["window"], case["sinks"])
        s["ws"] = torch.empty(256, dtype=torch.uint8, device=DEVICE)
        if case["kind"] == "quant":
            s["cache"] = oxd.KvPools(s["k"], s["v"], s["ks"], s["vs"])
    return s


def _prepare_prefill(case, seed):
    rng, g = np.random.default_rng(seed), _generator(seed)
    q, kv = np.asarray(_counts(case["q"])), np.asarray(_counts(case["kv"]))
    indptr, indices, last, pool = _tables(case, kv, kv - q, rng)
    qo = np.concatenate([[0], np.cumsum(q)]).astype(np.int32)
    n = int(qo[-1])
    s = dict(case=case, qo=_device(qo), indptr=_device(indptr), indices=_device(indices),
             last=_device(last), scale=1.0 / math.sqrt(128), q=_randn((n, case["hq"], 128), g),
             k=_fill(_pool_shape(case, pool, 128), g), v=_fill(_pool_shape(case, pool, 128), g))
    s["out"] = torch.empty_like(s["q"])
    s["lse"] = torch.empty((n, case["hq"]), device=DEVICE)
    if own:
        import paged_kv_decode_attn_gb300 as oxd

        desc = oxd.make_prefill_desc(len(q), case["hq"], case["hkv"], case["ps"], case["layout"], pool)
        s["plan"] = oxd.oxd_window_prefill_plan(desc, case["window"], case["sinks"], qo, indptr, last,
                                                torch.cuda.current_device())
        s["ws"] = torch.empty(s["plan"].workspace_bytes, dtype=torch.uint8, device=DEVICE)
        oxd.oxd_prefill_plan_bind_workspace(s["plan"], s["ws"])
    else:
        s["starts"] = [int(x) for x in indptr]
    return s


def _prepare_tables(case, seed):
    """Requests of a step: each holds `lengths` tokens with its new ones; its row of the page
    table lists the pages that it held before, and the rest come from the free list."""
    rng = np.random.default_rng(seed)
    b, ps = case["batch"], case["ps"]
    lengths = rng.integers(case["lo"], case["hi"] + 1, b)
    new = np.full(b, 1) if case["new"] == 1 else rng.integers(1, case["new"] + 1, b)
    new = np.minimum(new, lengths)
    held = -(-(lengths - new) // ps)
    most = -(-case["hi"] // ps)  # pages of a request at its longest: rows and buffers hold those
    width, pool = most + 2, b * most + 64
    order = rng.permutation(pool).astype(np.int32)
    rows = np.full((b, width), -1, np.int32)
    for i, end in enumerate(np.cumsum(held)):
        rows[i, :held[i]] = order[end - held[i]:end]
    free = order[int(held.sum()):]
    n_idx, n_tok = b * most, b * min(case["new"], case["hi"]) + 5
    s = dict(case=case, lengths=_device(lengths.astype(np.int32)), new=_device(new.astype(np.int32)),
             rows=_device(rows), held=_device(held.astype(np.int32)), free=_device(free),
             taken=torch.zeros(1, dtype=torch.int32, device=DEVICE))

    def out(n, dtype=torch.int32):
        return torch.full((n,), -9, dtype=dtype, device=DEVICE)

    s.update(indptr=out(b + 1), indices=out(n_idx), last=out(b), qo=out(b + 1), request=out(n_tok),
             positions=out(n_tok), slots=out(n_tok, torch.int64), held_out=out(b), taken_out=out(1),
             refcount=torch.zeros(pool, dtype=torch.int32, device=DEVICE))
    if own:
        import paged_kv_decode_attn_gb300 as oxd

        s["desc"] = oxd.make_build_tables_desc(
            batch=b, page_size=ps, row_pages=width, num_pages=pool, num_indices=n_idx,
            num_tokens=n_tok, num_free=len(free), window=case["window"], sinks=case["sinks"])
        s["ws"] = torch.empty(256, dtype=torch.uint8, device=DEVICE)
    return s


def prepare(case, seed):
    return {"decode": _prepare_decode, "quant": _prepare_decode, "prefill": _prepare_prefill,
            "tables": _prepare_tables}[case["kind"]](case, seed)


# ------------------------------------------------------------------ plain forms

def _dequantise(codes, scales):
    """codes u8 [..., 64], scales f16 [..., 4] -> f32 [..., 128]."""
    table = torch.tensor(LEVELS + tuple(-v for v in LEVELS), device=codes.device)
    pair = torch.stack([codes & 15, codes >> 4], -1).flatten(-2)
    return table[pair.int()] * scales.float().repeat_interleave(32, -1)


def _rows(s, name, page, slot):
    """The cached rows of tokens at (page, slot), f32 [..., heads, 128]."""
    pool = s[name].transpose(1, 2) if s["case"]["layout"] == "HND" else s[name]
    x = pool[page, slot]
    if s["case"]["kind"] != "quant":
        return x.float()
    return _dequantise(x, s[name + "s"].transpose(1, 2)[page, slot])


def _plain_decode(s):
    c = s["case"]
    b, hq, h, ps, w, sinks = c["batch"], c["hq"], c["hkv"], c["ps"], c["window"], c["sinks"]
    lo = (s["lengths"] - w).clamp(min=0)                   # first token of the window
    front = torch.minimum(lo, torch.full_like(lo, sinks))  # first tokens outside it
    count = front + s["lengths"] - lo
    n = min(c["hi"], w + sinks)
    i = torch.arange(n, device=DEVICE)
    out, lse = [], []
    step = max(1, (1 << 28) // (n * h * 128))
    for k0 in range(0, b, step):  # as many requests at once as memory holds
        part = slice(k0, k0 + step)
        token = torch.where(i < front[part, None], i, i - front[part, None] + lo[part, None])
        masked = i >= count[part, None]
        token = token.masked_fill(masked, 0)
        page = s["indices"][s["indptr"][:-1][part, None].long() + token // ps].long()
        masked = masked | (page < 0)
        page = page.clamp(min=0)
        k = _rows(s, "k", page, token % ps).permute(0, 2, 3, 1)
        q = s["q"][part].float().unflatten(1, (h, hq // h))
        x = (q @ k * s["scale"]).masked_fill(masked[:, None, None], -math.inf)
        top = x.amax(-1, keepdim=True)
        p = (x - top).exp()
        z = p.sum(-1, keepdim=True)
        v = _rows(s, "v", page, token % ps).transpose(1, 2)
        out.append((p @ v / z).flatten(1, 2))
        lse.append((top + z.log()).flatten(1))
    return {"out": torch.cat(out).to(torch.bfloat16), "lse": torch.cat(lse)}


def _plain_prefill(s):
    c = s["case"]
    hq, h, ps, w, sinks = c["hq"], c["hkv"], c["ps"], c["window"], c["sinks"]
    out, lse, at = [], [], 0
    for b, (n, length) in enumerate(zip(_counts(c["q"]), _counts(c["kv"]))):
        for i0 in range(0, n, 512):  # blocks of query tokens and the tokens that one of them sees
            m = min(512, n - i0)
            first = length - n + i0
            begin = max(0, first + 1 - w)
            token = torch.cat([torch.arange(min(sinks, begin), device=DEVICE),
                               torch.arange(begin, first + m, device=DEVICE)])
            page = s["indices"][s["starts"][b] + token // ps].long()
            k, v = (_rows(s, name, page, token % ps).transpose(0, 1) for name in ("k", "v"))
            q = s["q"][at + i0:at + i0 + m].float().unflatten(1, (h, hq // h)).permute(1, 2, 0, 3)
            pos = first + torch.arange(m, device=DEVICE)[:, None]
            seen = (token <= pos) & ((token > pos - w) | (token < sinks))
            x = q.flatten(1, 2) @ k.transpose(-1, -2) * s["scale"]
            x = x.unflatten(1, (hq // h, m)).masked_fill(~seen, -math.inf)
            top = x.amax(-1, keepdim=True)
            p = (x - top).exp()
            z = p.sum(-1, keepdim=True)
            o = (p.flatten(1, 2) @ v).unflatten(1, (hq // h, m)) / z
            out.append(o.permute(2, 0, 1, 3).flatten(1, 2))
            lse.append((top + z.log()).squeeze(-1).permute(2, 0, 1).flatten(1))
        at += n
    return {"out": torch.cat(out).to(torch.bfloat16), "lse": torch.cat(lse)}


def _plain_tables(s):
    c = s["case"]
    b, ps = c["batch"], c["ps"]
    lengths, new = s["lengths"].long(), s["new"].long()
    need = (lengths + ps - 1) // ps
    lack = (need - s["held"]).clamp(min=0)
    zero = torch.zeros(1, dtype=torch.int64, device=DEVICE)
    indptr = torch.cat([zero, need.cumsum(0)])
    qo = torch.cat([zero, new.cumsum(0)])
    first_free = s["taken"].long() + lack.cumsum(0) - lack

    def owners(ends, n):
        i = torch.arange(n, device=DEVICE)
        who = torch.searchsorted(ends[1:].contiguous(), i, right=True)
        return i, who.clamp(max=b - 1), who < b

    # pages of the tables: what a request holds, then what it takes
    i, who, there = owners(indptr, s["indices"].numel())
    j = i - indptr[who]
    taking = there & (j >= s["held"][who])
    page = torch.where(taking, s["free"][(first_free[who] + j - s["held"][who]).clamp(0, s["free"].numel() - 1)],
                       s["rows"][who, j.clamp(max=s["rows"].shape[1] - 1)])
    s["rows"][who[taking], j[taking]] = page[taking]
    s["refcount"][page[taking].long()] = 1
    if c["window"]:
        seen = lengths - new.clamp(min=1) + 1 - c["window"]  # the first token in a window
        page = torch.where((j * ps >= c["sinks"]) & ((j + 1) * ps <= seen[who]), -1, page)
    s["indices"].copy_(torch.where(there, page, s["indices"]))
    s["indptr"].copy_(indptr)
    s["last"].copy_(torch.where(need > 0, lengths - (need - 1) * ps, 0))
    s["qo"].copy_(qo)
    s["held_out"].copy_(torch.maximum(need, s["held"].long()))
    s["taken_out"].copy_(s["taken"] + lack.sum())
    # the new tokens
    i, who, there = owners(qo, s["request"].numel())
    pos = lengths[who] - new[who] + i - qo[who]
    at = s["rows"][who, (pos // ps).clamp(0, s["rows"].shape[1] - 1)].long() * ps + pos % ps
    s["request"].copy_(torch.where(there, who, -1))
    s["positions"].copy_(torch.where(there, pos, -1))
    s["slots"].copy_(torch.where(there, at, -1))
    return _tables_outputs(s)


def _tables_outputs(s):
    return {n: s[n] for n in ("indptr", "indices", "last", "qo", "request", "positions", "slots",
                              "rows", "held_out", "taken_out", "refcount")}


# ------------------------------------------------------------------ one pass

def _own_pass(s):
    import paged_kv_decode_attn_gb300 as oxd

    kind = s["case"]["kind"]
    if kind == "tables":
        oxd.oxd_build_tables(s["desc"], s["lengths"], s["new"], s["rows"], s["held"], s["held_out"],
                             s["free"], s["taken"], s["taken_out"], s["refcount"], s["indptr"],
                             s["indices"], s["last"], s["qo"], s["request"], s["positions"],
                             s["slots"], s["ws"])
        return _tables_outputs(s)
    if kind == "prefill":
        oxd.oxd_paged_prefill_run(s["plan"], s["q"], s["k"], s["v"], s["qo"], s["indptr"],
                                  s["indices"], s["last"], s["scale"], s["out"], s["lse"], s["ws"])
    elif kind == "quant":
        oxd.oxd_quant_window_decode(s["desc"], s["q"], s["cache"], s["indptr"], s["indices"],
                                    s["last"], s["scale"], s["out"], s["lse"], s["ws"])
    else:
        oxd.oxd_window_decode(s["desc"], s["q"], s["k"], s["v"], s["indptr"], s["indices"],
                              s["last"], s["scale"], s["out"], s["lse"], s["ws"])
    return {"out": s["out"], "lse": s["lse"]}


def run(state):
    if own:
        return _own_pass(state)
    return {"decode": _plain_decode, "quant": _plain_decode, "prefill": _plain_prefill,
            "tables": _plain_tables}[state["case"]["kind"]](state)


# ------------------------------------------------------------------ what a pass cannot do without

def work(case):
    kind = case["kind"]
    if kind == "tables":
        b, mean = case["batch"], (case["lo"] + case["hi"]) / 2
        pages = b * (mean / case["ps"] + 0.5)
        tokens = b * (1 if case["new"] == 1 else (1 + case["new"]) / 2)
        return {"bytes": pages * 8.0 + b * 28.0 + tokens * 16.0, "flops": 0.0}
    h, hq = case["hkv"], case["hq"]
    row = 2 * h * (72 if kind == "quant" else 256)
    if kind == "prefill":
        q, kv = np.asarray(_counts(case["q"])), np.asarray(_counts(case["kv"]))
        most = case["window"] + case["sinks"]
        pairs = sum(float(np.minimum(np.arange(l - n, l) + 1, most).sum()) for n, l in zip(q, kv))
        tokens = sum(min(l, n + most - 1) for n, l in zip(q, kv))
        return {"bytes": float(tokens * row + q.sum() * hq * 516), "flops": 512.0 * hq * pairs}
    lo, hi, most = case["lo"], case["hi"], case["window"] + case["sinks"]
    seen = float(np.minimum(np.arange(lo, hi + 1), most).mean()) * case["batch"]
    return {"bytes": seen * row + case["batch"] * hq * 516.0, "flops": 512.0 * hq * seen}


# ------------------------------------------------------------------ in 64 bits

def _exact_rows(s, name, request, length):
    """All rows of one request, f64 [length, heads, 128]; rows of pages not held are NaN."""
    c = s["case"]
    a, e = int(s["indptr"][request]), int(s["indptr"][request + 1])
    pages = s["indices"][a:e].long()
    x = s[name][pages.clamp(min=0)]
    if c["kind"] == "quant":
        codes = x.to(torch.int64)
        both = torch.stack((codes % 16, torch.div(codes, 16, rounding_mode="floor")), -1).flatten(-2)
        exponent, mantissa = torch.div(both, 2, rounding_mode="floor") % 4, (both % 2).double()
        size = torch.where(exponent == 0, 0.5 * mantissa,
                           (1 + 0.5 * mantissa) * torch.exp2(exponent.double() - 1))
        scale = s[name + "s"][pages.clamp(min=0)].double()
        if c["layout"] == "NHD":
            scale = scale.transpose(1, 2)
        x = ((1.0 - 2.0 * (both > 7)) * size).unflatten(-1, (4, 32)) * scale.unsqueeze(-1)
        x = x.flatten(-2)
    x = x.double()
    x[pages < 0] = math.nan
    if c["layout"] == "HND":
        x = x.transpose(1, 2)
    return x.flatten(0, 1)[:length]


def _exact_attention(s, q, k, v, first):
    """q f64 [n, Hq, 128] at positions first.. over rows [L, H, 128]: out and lse."""
    c = s["case"]
    n, group = q.shape[0], c["hq"] // c["hkv"]
    pos = torch.arange(first, first + n, device=DEVICE)
    j = torch.arange(k.shape[0], device=DEVICE)
    age = pos[:, None] - j
    seen = (age >= 0) & ((age < c["window"]) | (j < c["sinks"]))
    used = seen.any(0)
    seen, k, v = seen[:, used], k[used], v[used]
    out = torch.empty_like(q)
    lse = torch.empty(q.shape[:2], dtype=torch.float64, device=DEVICE)
    for head in range(c["hq"]):
        x = s["scale"] * (q[:, head] @ k[:, head // group].T)
        x = torch.where(seen, x, torch.full_like(x, -math.inf))
        lse[:, head] = torch.logsumexp(x, -1)
        out[:, head] = torch.softmax(x, -1) @ v[:, head // group]
    return out, lse


def _exact_tables(s):
    c = s["case"]
    ps = c["ps"]
    lengths, new, held = (s[n].tolist() for n in ("lengths", "new", "held"))
    rows, free = s["rows"].cpu().numpy().astype(np.int64), s["free"].cpu().numpy()
    indices = s["indices"].cpu().numpy().astype(np.int64)
    refcount = s["refcount"].cpu().numpy().astype(np.int64)
    request, positions, slots = (np.full(s["request"].numel(), -1, np.int64) for _ in range(3))
    indptr, qo, last, taken = [0], [0], [], int(s["taken"][0])
    for b, (length, n) in enumerate(zip(lengths, new)):
        pages = math.ceil(length / ps)
        for j in range(held[b], pages):
            rows[b, j] = free[taken]
            refcount[free[taken]] = 1
            taken += 1
        listed_pages = rows[b, :pages].copy()
        if c["window"]:
            oldest = length - max(n, 1) - c["window"] + 1
            for j in range(pages):
                if j * ps >= c["sinks"] and j * ps + ps - 1 < oldest:
                    listed_pages[j] = -1
        indices[indptr[b]:indptr[b] + pages] = listed_pages
        p = np.arange(length - n, length)
        request[qo[b]:qo[b] + n], positions[qo[b]:qo[b] + n] = b, p
        slots[qo[b]:qo[b] + n] = rows[b, p // ps] * ps + p % ps
        indptr.append(indptr[b] + pages)
        qo.append(qo[b] + n)
        last.append(length - (pages - 1) * ps if pages else 0)
        held[b] = max(held[b], pages)
    got = dict(indptr=indptr, indices=indices, last=last, qo=qo, request=request,
               positions=positions, slots=slots, rows=rows, held_out=held, taken_out=[taken],
               refcount=refcount)
    return {n: torch.as_tensor(np.asarray(x, np.int64), device=DEVICE) for n, x in got.items()}


def exact(case, seed):
    s = prepare(case, seed)
    if case["kind"] == "tables":
        return _exact_tables(s)
    q = s["q"].double()
    out, lse, at = [], [], 0
    counts = _counts(case["q"]) if case["kind"] == "prefill" else [1] * case["batch"]
    lengths = _counts(case["kv"]) if case["kind"] == "prefill" else s["lengths"].tolist()
    for b, (n, length) in enumerate(zip(counts, lengths)):
        k, v = (_exact_rows(s, name, b, length) for name in ("k", "v"))
        o, z = _exact_attention(s, q[at:at + n], k, v, length - n)
        out.append(o)
        lse.append(z)
        at += n
    return {"out": torch.cat(out), "lse": torch.cat(lse)}
