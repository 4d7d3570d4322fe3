"""What the operators of the 4-bit paged KV cache cost, against their plain forms.

Four operators around the paged cache are measured:

* ``decode``  one decode step over a cache held in 4 bits (``oxd_quant_decode_run``);
* ``append4`` rotary embedding of new tokens and their K/V rows written into 4-bit pages
  (``oxd_quant_rope_append``), the touched pages read back as bf16 (``oxd_copy_pages``);
* ``append``  rotary embedding with one or several position axes and the append into bf16
  pages (``oxd_rope_axes_append``);
* ``copy`` / ``pack``  pages copied inside a pool, packed into 4 bits and unpacked
  (``oxd_copy_pages``).

The 4-bit format: the 128 values of one (token, KV head) are four groups of 32. A group's
scale is the f16 nearest to amax / 6 (at most 10912), a value's code the e2m1 number
(0, 0.5, 1, 1.5, 2, 3, 4, 6 and their negatives) nearest to value / scale, ties to the even
code, at most 6 in size. Two codes a byte, the even column in the low half. Codes are
[pages, page_size, heads, 64] (NHD) or [pages, heads, page_size, 64] (HND), scales
[pages, heads, page_size, 4] f16 in both.
"""
import math

import numpy as np
import torch

own = False

DEVICE = "cuda"
THETA = 10000.0
SECTIONS = (16, 24, 24)  # rotary pairs of the time, height and width axes
LEVELS = (0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0)


# ------------------------------------------------------------------ cases

def listed():
    return [
        # one request of a small model, a short chat turn: latency
        dict(name="decode_mha8_b1", kind="decode", batch=1, hq=8, hkv=8, ps=16, layout="NHD",
             dist="uniform", lo=512, hi=512, sigma=1.0),
        # a serving batch with the lengths a log-normal gives (median 2048)
        dict(name="decode_gqa4_b128", kind="decode", batch=128, hq=32, hkv=8, ps=16, layout="HND",
             dist="lognormal", lo=128, hi=8192, sigma=1.0),
        # few long documents, one KV head for 32 query heads
        dict(name="decode_mqa32_b16", kind="decode", batch=16, hq=32, hkv=1, ps=64, layout="NHD",
             dist="uniform", lo=32768, hi=32768, sigma=1.0),
        # the largest batch of the decode benchmark
        dict(name="decode_gqa8_b256", kind="decode", batch=256, hq=64, hkv=8, ps=16, layout="NHD",
             dist="uniform", lo=128, hi=16384, sigma=1.5),
        # one new token for each request of a decode batch
        dict(name="append4_step_b32", kind="append4", batch=32, tokens=1, hq=32, hkv=8, ps=16,
             layout="NHD", axes=1, start=4095),
        # prompts of odd length with images, on three position axes
        dict(name="append4_images_b4", kind="append4", batch=4, tokens=1223, hq=32, hkv=8, ps=16,
             layout="HND", axes=3, start=0),
        # a long prompt in one call
        dict(name="append4_prompt_b8", kind="append4", batch=8, tokens=2048, hq=32, hkv=8, ps=16,
             layout="NHD", axes=1, start=0),
        # one new token for each request, on three position axes
        dict(name="append_step_b64", kind="append", batch=64, tokens=1, hq=32, hkv=8, ps=16,
             layout="NHD", axes=3, start=511),
        # prompts with images into bf16 pages
        dict(name="append_images_b8", kind="append", batch=8, tokens=2048, hq=32, hkv=8, ps=16,
             layout="NHD", axes=3, start=0),
        # a fork: the last pages of eight sequences made private
        dict(name="copy_fork_8", kind="copy", pairs=8, pages=512, hkv=8, ps=16, layout="NHD"),
        # a compaction: live pages moved into the holes of a large pool
        dict(name="copy_move_4096", kind="copy", pairs=4096, pages=12288, hkv=8, ps=16,
             layout="HND"),
        # the pages of prefilled prompts packed into 4 bits, and unpacked for another prefill
        dict(name="pack_4096", kind="pack", pairs=4096, pages=4608, hkv=8, ps=16, layout="NHD"),
    ]


def _log_uniform(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    kind = rng.choice(["decode", "decode", "append4", "append", "copy", "pack"])
    ps = rng.choice([8, 16, 32, 64])
    layout = rng.choice(["NHD", "HND"])
    hkv = rng.choice([1, 2, 3, 4, 8, 16])
    if kind == "decode":
        group = rng.choice([1, 2, 4, 5, 8, 16, 32])
        batch = _log_uniform(rng, 1, 256)
        most = max(2, min(32768, 9_000_000 // (batch * hkv)))
        hi = _log_uniform(rng, 2, most)
        lo = rng.choice([1, max(1, hi // 4), hi])
        return dict(kind="decode", batch=batch, hq=group * hkv, hkv=hkv, ps=ps, layout=layout,
                    dist="uniform", lo=lo, hi=hi, sigma=rng.choice([0.5, 1.0, 1.5]))
    if kind in ("append4", "append"):
        batch = _log_uniform(rng, 1, 128)
        tokens = _log_uniform(rng, 1, max(1, 16384 // batch))
        return dict(kind=kind, batch=batch, tokens=tokens, hq=rng.choice([1, 2, 4, 7, 8]) * hkv,
                    hkv=hkv, ps=ps, layout=layout, axes=rng.choice([1, 3]),
                    start=rng.choice([0, 1, rng.randrange(0, 4096)]))
    pairs = _log_uniform(rng, 1, 65536 // ps // hkv)
    return dict(kind=kind, pairs=pairs, pages=2 * pairs + rng.randrange(1, 64), hkv=hkv, ps=ps,
                layout=layout)


# ------------------------------------------------------------------ the format, plainly

def _round_bf16(x):
    """f64 values rounded to 8 significant bits, ties to even, as bf16."""
    m, e = torch.frexp(x)
    return torch.ldexp(torch.round(m * 256.0), e - 8).to(torch.bfloat16)


def _quantise(x):
    """bf16 rows [..., 128] -> codes u8 [..., 64], scales f16 [..., 4]."""
    g = x.float().unflatten(-1, (4, 32))
    scale = (g.abs().amax(-1) / 6.0).clamp(max=10912.0).half()
    s = scale.float().unsqueeze(-1)
    y = torch.where(s > 0, g / s, torch.zeros_like(g))
    a = y.abs()
    code = ((a > 0.25).byte() + (a >= 0.75).byte() + (a > 1.25).byte() + (a >= 1.75).byte()
            + (a > 2.5).byte() + (a >= 3.5).byte() + (a > 5.0).byte() + 8 * (y < 0).byte())
    code = code.flatten(-2)
    return code[..., 0::2] + 16 * code[..., 1::2], scale


def _dequantise(codes, scales):
    """codes u8 [..., 64], scales f16 [..., 4] -> f32 [..., 128]."""
    table = torch.tensor(LEVELS + tuple(-v for v in LEVELS), device=codes.device)
    pair = torch.stack([codes & 15, codes >> 4], -1).flatten(-2)
    return table[pair.int()] * scales.float().repeat_interleave(32, -1)


def _scales_as_codes(scales, layout):
    """Scales [pages, heads, page_size, 4] in the order of the codes' first three axes."""
    return scales.transpose(1, 2) if layout == "NHD" else scales


# ------------------------------------------------------------------ inputs

def _generator(seed):
    return torch.Generator(device=DEVICE).manual_seed(seed)


def _randn(shape, g, sigma=1.0):
    return torch.randn(shape, generator=g, device=DEVICE).mul_(sigma).to(torch.bfloat16)


def _tables(pages, rng, extra=0):
    """Page lists of requests with `pages` pages each: indptr, indices over a shuffled pool."""
    indptr = np.concatenate([[0], np.cumsum(pages)]).astype(np.int32)
    pool = int(indptr[-1]) + extra
    return indptr, rng.permutation(pool)[:indptr[-1]].astype(np.int32), pool


def _pool_shape(case, pages, width):
    ps, h = case["ps"], case["hkv"]
    return (pages, ps, h, width) if case["layout"] == "NHD" else (pages, h, ps, width)


def _lengths(case, rng):
    b, lo, hi = case["batch"], case["lo"], case["hi"]
    if case["dist"] == "lognormal":
        return np.clip(np.rint(np.exp(rng.normal(math.log(2048), 1.0, b))), lo, hi).astype(np.int64)
    return rng.integers(lo, hi + 1, b)


def _packed_pool(case, pages, g):
    """A pool of normal values held in 4 bits: codes and scales."""
    codes = torch.empty(_pool_shape(case, pages, 64), dtype=torch.uint8, device=DEVICE)
    scales = torch.empty((pages, case["hkv"], case["ps"], 4), dtype=torch.float16, device=DEVICE)
    step = max(1, (1 << 26) // (case["ps"] * case["hkv"] * 128))
    for p in range(0, pages, step):
        n = min(step, pages - p)
        codes[p:p + n], s = _quantise(_randn(_pool_shape(case, n, 128), g, case["sigma"]))
        scales[p:p + n] = s.transpose(1, 2) if case["layout"] == "NHD" else s
    return codes, scales


def _device(a):
    return torch.as_tensor(a, device=DEVICE)


def _prepare_decode(case, seed):
    rng, g = np.random.default_rng(seed), _generator(seed)
    lengths = _lengths(case, rng)
    ps = case["ps"]
    pages = -(-lengths // ps)
    indptr, indices, pool = _tables(pages, rng)
    last = (lengths - (pages - 1) * ps).astype(np.int32)
    s = dict(case=case, lengths=_device(lengths), indptr=_device(indptr), indices=_device(indices),
             last=_device(last), scale=1.0 / math.sqrt(128),
             q=_randn((case["batch"], case["hq"], 128), g, case["sigma"]))
    s["k"], s["ks"] = _packed_pool(case, pool, g)
    s["v"], s["vs"] = _packed_pool(case, pool, g)
    s["out"] = torch.empty_like(s["q"])
    s["lse"] = torch.empty((case["batch"], case["hq"]), device=DEVICE)
    if own:
        import paged_kv_decode_attn_gb300 as oxd

        desc = oxd.make_desc(case["batch"], case["hq"], case["hkv"], ps, case["layout"], pool)
        s["plan"] = oxd.oxd_quant_decode_plan(desc, indptr, last, torch.cuda.current_device())
        s["ws"] = torch.empty(s["plan"].workspace_bytes, dtype=torch.uint8, device=DEVICE)
        s["cache"] = oxd.KvPools(s["k"], s["v"], s["ks"], s["vs"])
        oxd.oxd_plan_bind_workspace(s["plan"], s["ws"])
    else:
        s["page_list"] = np.split(indices, indptr[1:-1])
    return s


def _axis_positions(case, pos):
    """[axes, T]: text counts on all axes; from position 16 on, spans of 512 tokens in turn are
    images of 32 columns (time stands, height and width run) and text."""
    if case["axes"] == 1:
        return pos[None]
    span, at = (pos - 16) // 512, (pos - 16) % 512
    image = (pos >= 16) & (span % 2 == 0)
    base = pos - np.where(image, at, 0)
    return np.stack([np.where(image, base, pos), np.where(image, base + at // 32, pos),
                     np.where(image, base + at % 32, pos)])


def _prepare_append(case, seed):
    rng, g = np.random.default_rng(seed), _generator(seed)
    b, n, ps, h = case["batch"], case["tokens"], case["ps"], case["hkv"]
    first = np.maximum(0, case["start"] - np.arange(b) * 37 % 64)  # requests end at different slots
    ends = first + n
    indptr, indices, pool = _tables(-(-ends // ps), rng)
    request = np.repeat(np.arange(b), n)
    pos = (first[:, None] + np.arange(n)).reshape(-1)
    s = dict(case=case, request=_device(request.astype(np.int32)), pos=_device(pos.astype(np.int32)),
             rope=_device(_axis_positions(case, pos).astype(np.int32)), indptr=_device(indptr),
             indices=_device(indices), refcount=torch.ones(pool, dtype=torch.int32, device=DEVICE),
             q=_randn((b * n, case["hq"], 128), g), k=_randn((b * n, h, 128), g),
             v=_randn((b * n, h, 128), g))
    s["q_out"] = torch.empty_like(s["q"])
    if case["kind"] == "append":
        s["k_pages"] = torch.zeros(_pool_shape(case, pool, 128), dtype=torch.bfloat16, device=DEVICE)
        s["v_pages"] = torch.zeros_like(s["k_pages"])
    else:
        for name in ("k", "v"):
            s[name + "_codes"] = torch.zeros(_pool_shape(case, pool, 64), dtype=torch.uint8, device=DEVICE)
            s[name + "_scales"] = torch.zeros((pool, h, ps, 4), dtype=torch.float16, device=DEVICE)
        touched = np.unique(indices[indptr[request] + pos // ps])
        s["touched"] = _device(touched)
        s["rows"] = torch.arange(len(touched), dtype=torch.int32, device=DEVICE)
        s["k_read"] = torch.empty(_pool_shape(case, len(touched), 128), dtype=torch.bfloat16, device=DEVICE)
        s["v_read"] = torch.empty_like(s["k_read"])
    if own:
        import paged_kv_decode_attn_gb300 as oxd

        s["desc"] = oxd.make_axes_append_desc(b * n, b, case["hq"], h, ps, case["layout"], pool,
                                              len(indices), rope_theta=THETA,
                                              sections=SECTIONS if case["axes"] == 3 else (64,))
        s["ws"] = torch.empty(256, dtype=torch.uint8, device=DEVICE)
        if case["kind"] == "append4":
            s["cache"] = oxd.KvPools(s["k_codes"], s["v_codes"], s["k_scales"], s["v_scales"])
            s["read"] = oxd.KvPools(s["k_read"], s["v_read"])
            s["read_desc"] = oxd.make_copy_pages_desc(
                len(touched), h, ps, src_format="e2m1", src_layout=case["layout"], src_num_pages=pool,
                dst_format="bf16", dst_layout=case["layout"], dst_num_pages=len(touched))
    return s


def _prepare_pages(case, seed):
    rng, g = np.random.default_rng(seed), _generator(seed)
    n, pages, h, ps = case["pairs"], case["pages"], case["hkv"], case["ps"]
    order = rng.permutation(pages).astype(np.int32)
    s = dict(case=case, src=_device(order[:n]), k=_randn(_pool_shape(case, pages, 128), g),
             v=_randn(_pool_shape(case, pages, 128), g))
    if case["kind"] == "copy":
        s["dst"] = _device(order[n:2 * n])
        s["refcount"] = torch.ones(pages, dtype=torch.int32, device=DEVICE)
    else:
        s["dst"] = _device(rng.permutation(n).astype(np.int32))
        for name in ("k", "v"):
            s[name + "_codes"] = torch.zeros(_pool_shape(case, n, 64), dtype=torch.uint8, device=DEVICE)
            s[name + "_scales"] = torch.zeros((n, h, ps, 4), dtype=torch.float16, device=DEVICE)
            s[name + "_read"] = torch.empty(_pool_shape(case, n, 128), dtype=torch.bfloat16, device=DEVICE)
    if own:
        import paged_kv_decode_attn_gb300 as oxd

        def desc(src, src_pages, dst, dst_pages):
            return oxd.make_copy_pages_desc(n, h, ps, src_format=src, src_layout=case["layout"],
                                            src_num_pages=src_pages, dst_format=dst,
                                            dst_layout=case["layout"], dst_num_pages=dst_pages)

        s["ws"] = torch.empty(256, dtype=torch.uint8, device=DEVICE)
        s["pools"] = oxd.KvPools(s["k"], s["v"])
        if case["kind"] == "copy":
            s["desc"] = desc("bf16", pages, "bf16", pages)
        else:
            s["pack_desc"] = desc("bf16", pages, "e2m1", n)
            s["unpack_desc"] = desc("e2m1", n, "bf16", n)
            s["cache"] = oxd.KvPools(s["k_codes"], s["v_codes"], s["k_scales"], s["v_scales"])
            s["read"] = oxd.KvPools(s["k_read"], s["v_read"])
    return s


def prepare(case, seed):
    return {"decode": _prepare_decode, "append4": _prepare_append, "append": _prepare_append,
            "copy": _prepare_pages, "pack": _prepare_pages}[case["kind"]](case, seed)


# ------------------------------------------------------------------ plain forms

def _gather(codes, scales, pages, layout):
    """The tokens of page lists [n, p] as f32 [n, heads, p * page_size, 128]."""
    x = _dequantise(codes[pages], _scales_as_codes(scales, layout)[pages])
    x = x.permute(0, 3, 1, 2, 4) if layout == "NHD" else x.permute(0, 2, 1, 3, 4)
    return x.flatten(2, 3)


def _plain_decode(s):
    c = s["case"]
    b, hq, h, ps = c["batch"], c["hq"], c["hkv"], c["ps"]
    lists = s["page_list"]
    longest = max(len(p) for p in lists)
    table = np.zeros((b, longest), np.int64)
    for i, p in enumerate(lists):
        table[i, :len(p)] = p
    table = _device(table)
    step = max(1, (1 << 29) // (longest * ps * h * 128))
    out, lse = [], []
    for i in range(0, b, step):  # as many requests at once as memory holds
        pages = table[i:i + step]
        k = _gather(s["k"], s["ks"], pages, c["layout"])
        q = s["q"][i:i + step].float().unflatten(1, (h, hq // h))
        x = q @ k.transpose(-1, -2) * s["scale"]
        masked = torch.arange(x.shape[-1], device=DEVICE) >= s["lengths"][i:i + step, None]
        x = x.masked_fill(masked[:, None, None], -math.inf)
        m = x.amax(-1, keepdim=True)
        p = (x - m).exp()
        z = p.sum(-1, keepdim=True)
        v = _gather(s["v"], s["vs"], pages, c["layout"])
        out.append((p @ v / z).flatten(1, 2))
        lse.append((m + z.log()).flatten(1))
    return {"out": torch.cat(out).to(torch.bfloat16), "lse": torch.cat(lse)}


def _pair_axis(case, device):
    sections = SECTIONS if case["axes"] == 3 else (64,)
    return torch.repeat_interleave(torch.arange(len(sections), device=device),
                                   torch.tensor(sections, device=device))


def _plain_rotate(case, x, rope):
    """Split-half rotary embedding in f64 (angles of far positions, codes next to a border)."""
    freq = THETA ** (-torch.arange(64, dtype=torch.float64, device=x.device) / 64.0)
    angle = rope[_pair_axis(case, x.device)].T.double() * freq
    cos, sin = angle.cos().unsqueeze(1), angle.sin().unsqueeze(1)
    a, b = x[..., :64].double(), x[..., 64:].double()
    return _round_bf16(torch.cat([a * cos - b * sin, b * cos + a * sin], -1))


def _write_rows(case, pages, rows, page, slot):
    if case["layout"] == "NHD":
        pages[page, slot] = rows
    else:
        pages[page, :, slot] = rows


def _plain_append(s):
    c = s["case"]
    page = s["indices"][(s["indptr"][s["request"].long()] + s["pos"] // c["ps"]).long()].long()
    slot = (s["pos"] % c["ps"]).long()
    q = _plain_rotate(c, s["q"], s["rope"])
    k = _plain_rotate(c, s["k"], s["rope"])
    if c["kind"] == "append":
        _write_rows(c, s["k_pages"], k, page, slot)
        _write_rows(c, s["v_pages"], s["v"], page, slot)
        return {"q": q, "k": s["k_pages"], "v": s["v_pages"]}
    got = {"q": q}
    for name, rows in (("k", k), ("v", s["v"])):
        codes, scales = _quantise(rows)
        _write_rows(c, s[name + "_codes"], codes, page, slot)
        s[name + "_scales"][page, :, slot] = scales
        at = s["touched"].long()
        got[name] = _dequantise(s[name + "_codes"][at],
                                _scales_as_codes(s[name + "_scales"], c["layout"])[at]).to(torch.bfloat16)
    return got


def _plain_pages(s):
    c = s["case"]
    src, dst = s["src"].long(), s["dst"].long()
    if c["kind"] == "copy":
        s["k"][dst] = s["k"][src]
        s["v"][dst] = s["v"][src]
        return {"k": s["k"], "v": s["v"]}
    got = {}
    for name in ("k", "v"):
        codes, scales = _quantise(s[name][src])
        s[name + "_codes"][dst] = codes
        s[name + "_scales"][dst] = _scales_as_codes(scales, c["layout"])
        back = _dequantise(s[name + "_codes"][dst], _scales_as_codes(s[name + "_scales"], c["layout"])[dst])
        s[name + "_read"][dst] = back.to(torch.bfloat16)
        got[name] = s[name + "_read"]
    return got


# ------------------------------------------------------------------ one pass

def _own_pass(s):
    import paged_kv_decode_attn_gb300 as oxd

    kind = s["case"]["kind"]
    if kind == "decode":
        oxd.oxd_quant_decode_run(s["plan"], s["q"], s["cache"], s["indptr"], s["indices"], s["last"],
                                 s["scale"], s["out"], s["lse"], s["ws"])
        return {"out": s["out"], "lse": s["lse"]}
    if kind == "append":
        oxd.oxd_rope_axes_append(s["desc"], s["q"], s["k"], s["v"], s["request"], s["pos"], s["rope"],
                                 s["indptr"], s["indices"], s["refcount"], s["q_out"], s["k_pages"],
                                 s["v_pages"], s["ws"])
        return {"q": s["q_out"], "k": s["k_pages"], "v": s["v_pages"]}
    if kind == "append4":
        oxd.oxd_quant_rope_append(s["desc"], s["q"], s["k"], s["v"], s["request"], s["pos"], s["rope"],
                                  s["indptr"], s["indices"], s["refcount"], s["q_out"], s["cache"],
                                  s["ws"])
        oxd.oxd_copy_pages(s["read_desc"], s["cache"], s["read"], s["touched"], s["rows"], None, s["ws"])
        return {"q": s["q_out"], "k": s["k_read"], "v": s["v_read"]}
    if kind == "copy":
        oxd.oxd_copy_pages(s["desc"], s["pools"], s["pools"], s["src"], s["dst"], s["refcount"], s["ws"])
        return {"k": s["k"], "v": s["v"]}
    oxd.oxd_copy_pages(s["pack_desc"], s["pools"], s["cache"], s["src"], s["dst"], None, s["ws"])
    oxd.oxd_copy_pages(s["unpack_desc"], s["cache"], s["read"], s["dst"], s["dst"], None, s["ws"])
    return {"k": s["k_read"], "v": s["v_read"]}


def run(state):
    if own:
        return _own_pass(state)
    return {"decode": _plain_decode, "append4": _plain_append, "append": _plain_append,
            "copy": _plain_pages, "pack": _plain_pages}[state["case"]["kind"]](state)


# ------------------------------------------------------------------ what a pass cannot do without

def work(case):
    h, ps = case["hkv"], case["ps"]
    row4, row16 = h * 72, h * 256  # bytes of one token's K (or V) rows in 4 and in 16 bits
    if case["kind"] == "decode":
        b, hq = case["batch"], case["hq"]
        mean = (case["lo"] + case["hi"]) / 2 if case["dist"] == "uniform" else 2740.0
        tokens = b * mean
        return {"bytes": tokens * 2 * row4 + b * hq * (128 * 4 + 4) + tokens / ps * 4,
                "flops": 4.0 * 128 * hq * tokens}
    if case["kind"] in ("append4", "append"):
        t = case["batch"] * case["tokens"]
        rows = t * (case["hq"] * 512 + 2 * row16)
        flops = 6.0 * 64 * t * (case["hq"] + h)
        if case["kind"] == "append":
            return {"bytes": rows + t * 2 * row16, "flops": flops}
        pages = case["batch"] * math.ceil(case["tokens"] / ps)  # read back as bf16
        return {"bytes": rows + t * 2 * row4 + pages * ps * 2 * (row4 + row16),
                "flops": flops + 6.0 * 256 * t * h}
    n = case["pairs"] * ps * 2
    if case["kind"] == "copy":
        return {"bytes": n * 2.0 * row16, "flops": 0.0}
    return {"bytes": n * 2.0 * (row16 + row4), "flops": 6.0 * n * h * 128}


# ------------------------------------------------------------------ in 64 bits

def _exact_levels(codes, scales):
    """Codes and scales (already in one order) as f64 values."""
    c = codes.to(torch.int32)
    both = torch.empty(codes.shape[:-1] + (128,), dtype=torch.int32, device=codes.device)
    both[..., 0::2], both[..., 1::2] = c % 16, c // 16
    exponent, mantissa = (both // 2) % 4, both % 2
    size = torch.where(exponent == 0, mantissa * 0.5,
                       (1 + mantissa * 0.5) * torch.exp2((exponent - 1).double()))
    value = torch.where(both >= 8, -size, size)
    return (value.unflatten(-1, (4, 32)) * scales.double().unsqueeze(-1)).flatten(-2)


def _exact_hold(x):
    """What f64 rows [..., 128] of bf16 values become in 4 bits."""
    g = x.unflatten(-1, (4, 32))
    scale = torch.minimum(g.abs().amax(-1, keepdim=True) / 6, torch.tensor(10912.0, device=x.device,
                                                                           dtype=torch.float64)).half().double()
    size = torch.where(scale > 0, g.abs() / scale, torch.zeros_like(g))
    # the spacing of e2m1 numbers is half below 2, one below 4, two above
    step = torch.where(size < 1.75, 0.5, torch.where(size < 3.5, 1.0, 2.0)).double()
    return (torch.copysign((torch.round(size / step) * step).clamp(max=6), g) * scale).flatten(-2)


def _exact_decode(s):
    c = s["case"]
    g = c["hq"] // c["hkv"]
    out = torch.empty(s["q"].shape, dtype=torch.float64, device=DEVICE)
    lse = torch.empty(s["lse"].shape, dtype=torch.float64, device=DEVICE)
    indptr, lengths = s["indptr"].tolist(), s["lengths"].tolist()
    for b in range(c["batch"]):
        at = s["indices"][indptr[b]:indptr[b + 1]].long()
        order = (2, 0, 1, 3) if c["layout"] == "NHD" else (1, 0, 2, 3)
        k, v = (_exact_levels(s[n][at], _scales_as_codes(s[n + "s"], c["layout"])[at])
                .permute(order).flatten(1, 2)[:, :lengths[b]] for n in ("k", "v"))
        x = torch.einsum("hgd,htd->hgt", s["q"][b].double().reshape(c["hkv"], g, 128), k) * s["scale"]
        top = torch.logsumexp(x, -1, keepdim=True)
        out[b] = torch.einsum("hgt,htd->hgd", torch.exp(x - top), v).reshape(c["hq"], 128)
        lse[b] = top.reshape(-1)
    return {"out": out, "lse": lse}


def _exact_turn(case, x, rope):
    i = torch.arange(64, dtype=torch.float64, device=x.device)
    axis = [0] * 64 if case["axes"] == 1 else [0] * SECTIONS[0] + [1] * SECTIONS[1] + [2] * SECTIONS[2]
    angle = rope.double()[torch.tensor(axis, device=x.device)] * torch.pow(THETA, -2 * i / 128)[:, None]
    turn = torch.polar(torch.ones_like(angle), angle).T.unsqueeze(1)
    z = torch.complex(x[..., :64].double(), x[..., 64:].double()) * turn
    return torch.cat([z.real, z.imag], -1)


def _exact_append(s):
    c = s["case"]
    which = s["indptr"].long()[s["request"].long()] + torch.div(s["pos"].long(), c["ps"], rounding_mode="floor")
    page, slot = s["indices"].long()[which], s["pos"].long() % c["ps"]
    k, v = _exact_turn(c, s["k"], s["rope"]), s["v"].double()
    if c["kind"] == "append":
        pools = [s["k_pages"].double(), s["v_pages"].double()]
    else:
        # to the bf16 number nearest, then to 4 bits; rows in the order of the pages read back
        ulp = torch.exp2(torch.floor(torch.log2(k.abs().clamp(min=1e-30))) - 7)
        k, v = _exact_hold(torch.round(k / ulp) * ulp), _exact_hold(v)
        pools = [torch.zeros(s["k_read"].shape, dtype=torch.float64, device=DEVICE) for _ in "kv"]
        page = torch.searchsorted(s["touched"].long(), page)
    for pool, rows in zip(pools, (k, v)):
        (pool if c["layout"] == "NHD" else pool.transpose(1, 2))[page, slot] = rows
    return {"q": _exact_turn(c, s["q"], s["rope"]), "k": pools[0], "v": pools[1]}


def _exact_pages(s):
    src, dst = s["src"].long(), s["dst"].long()
    got = {}
    for n in ("k", "v"):
        if s["case"]["kind"] == "copy":
            x = s[n].double()
            x[dst] = s[n].double()[src]
        else:
            x = torch.empty(s[n + "_read"].shape, dtype=torch.float64, device=DEVICE)
            x[dst] = _exact_hold(s[n][src].double())
        got[n] = x
    return got


def exact(case, seed):
    s = prepare(case, seed)
    return {"decode": _exact_decode, "append4": _exact_append, "append": _exact_append,
            "copy": _exact_pages, "pack": _exact_pages}[case["kind"]](s)
