"""Cases of the paged latent-cache operators: attention of new tokens over pages (whole context, or a sliding
window with sinks) and the cache's write and read-back, in plain torch form and as the library's calls.

A case's "kind" is "attn" (mla_attn_paged) or "cache" (mla_paged_append followed by mla_paged_gather).  A batch has
"batch" sequences; sequence b holds len[b] rows (len_lo..len_hi) of which the last new[b] (new_lo..new_hi) are
this call's tokens.  "cache" is the page type: "f16" (576 fp16 a row) or "e4m3" (656 bytes a row: 512 codes, 64
fp16, 16 power-of-two scales); "page" the rows of a page; "window" 0 for the whole context.
"""
import math
import random

import numpy as np
import torch

own = False

LAT, ROPE, ROW, ROW8 = 512, 64, 576, 656
SCALE = 1.0 / math.sqrt(192.0)
FREQ_BASE, FREQ_SCALE = 10000.0, 0.025


def _attn(name, cache, heads, batch, new, length, page, window=0, sinks=0):
    return dict(name=name, kind="attn", cache=cache, heads=heads, batch=batch, new_lo=new[0], new_hi=new[1],
                len_lo=length[0], len_hi=length[1], page=page, window=window, sinks=sinks)


def _cache(name, cache, batch, new, length, page, extra):
    return dict(name=name, kind="cache", cache=cache, batch=batch, new_lo=new[0], new_hi=new[1], len_lo=length[0],
                len_hi=length[1], page=page, extra=extra)


def listed():
    return [
        # one user's next token, 16 heads, a short context: latency
        _attn("token_b1_h16", "f16", 16, 1, (1, 1), (257, 257), 64),
        # a serving batch's next tokens, 128 heads, contexts of 4K to 32K
        _attn("tokens_b32_h128", "f16", 128, 32, (1, 1), (4096, 32768), 64),
        # long contexts in an 8-bit cache
        _attn("tokens_b8_h128_e4m3", "e4m3", 128, 8, (1, 1), (98304, 98304), 128),
        # prompts of several users in one call, 16 heads, small pages, odd lengths
        _attn("chunks_b4_h16", "f16", 16, 4, (301, 1531), (301, 4099), 16),
        # a chunk of a long prompt, 128 heads
        _attn("chunk_h128_at32k", "f16", 128, 1, (512, 512), (33280, 33280), 64),
        # ragged chunks behind an 8-bit prefix (prefix cache), 64 heads
        _attn("chunks_b3_h64_e4m3", "e4m3", 64, 3, (77, 500), (2000, 9001), 32),
        # endless generation: a window of 4096 rows and four sinks over contexts of up to 64K
        _attn("window_tokens_b64_h128", "f16", 128, 64, (1, 1), (5000, 65536), 64, 4096, 4),
        # prompt chunks under a window, an 8-bit cache
        _attn("window_chunks_b2_h128_e4m3", "e4m3", 128, 2, (200, 600), (6000, 20000), 64, 1000, 16),
        # the cache side of one decode step: 64 new rows, written and read back
        _cache("rows_b64", "f16", 64, (1, 1), (1000, 65536), 64, 0),
        # the cache side of a chunked prefill: new rows written, the whole prefix read back
        _cache("rows_chunks_e4m3", "e4m3", 4, (700, 2048), (9001, 20000), 32, 6001),
        # a long prompt's rows into an 8-bit cache and back, and the same in 16 bits
        _cache("rows_98304_e4m3", "e4m3", 1, (98304, 98304), (98304, 98304), 64, 0),
        _cache("rows_98304_f16", "f16", 1, (98304, 98304), (98304, 98304), 128, 0),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    cache, page = rng.choice(("f16", "e4m3")), rng.choice((16, 32, 64, 128, 256))
    if rng.random() < 0.3:
        batch = _log(rng, 1, 64)
        new = _log(rng, 1, max(1, 98304 // batch))
        extra = rng.choice((0, _log(rng, 1, 8192)))
        length = new + extra + rng.randrange(0, 30000)
        c = _cache(None, cache, batch, (max(1, new - new // 5), new), (max(new + extra, length - length // 4), length),
                   page, extra)
        del c["name"]
        return c
    heads = 16 * rng.randint(1, 8)
    if rng.random() < 0.5:
        batch, new = _log(rng, 1, 64), 1
        hi = _log(rng, 16, 65536)
        hi = min(hi, 590000 * 2 // batch)
    else:
        batch = rng.randint(1, 6)
        new = _log(rng, 2, 2048)
        new = min(new, 3 * 10 ** 6 // (heads * batch))
        hi = new + _log(rng, 1, 32768)
        hi = max(new, min(hi, 2 * 10 ** 9 // (heads * batch * new)))
    window = _log(rng, 32, 8192) if rng.random() < 0.5 else 0
    sinks = rng.choice((0, 1, 4, 64, 100)) if window else 0
    c = _attn(None, cache, heads, batch, (max(1, new // 3), new), (max(new, hi // 4), max(new, hi)), page, window, sinks)
    del c["name"]
    return c


def _lengths(case):
    """new[b] and len[b]: spread over the case's ranges, the same for every seed; both ends are among them."""
    rng = random.Random("%(batch)d %(new_lo)d %(new_hi)d %(len_lo)d %(len_hi)d" % case)
    new = [rng.randint(case["new_lo"], case["new_hi"]) for _ in range(case["batch"])]
    length = [rng.randint(case["len_lo"], case["len_hi"]) for _ in range(case["batch"])]
    new[-1], length[-1] = case["new_hi"], case["len_hi"]
    if case["batch"] > 1:
        new[0], length[0] = case["new_lo"], case["len_lo"]
    return new, [max(n + case.get("extra", 0), l) for n, l in zip(new, length)]


def _quantise(x):
    """[..., 512] fp32 -> e4m3 codes (uint8) and one scale byte for 32 values: the smallest 2^(s - 127) in
    [2^-15, 2^7] with amax <= 448 * 2^(s - 127)."""
    x = x.unflatten(-1, (16, 32))
    m, e = torch.frexp(x.abs().amax(-1))
    e = torch.where(m <= 0.875, e - 9, e - 8)
    e = torch.where(m == 0, torch.full_like(e, -15), e).clamp(-15, 7)
    codes = torch.ldexp(x, -e[..., None]).to(torch.float8_e4m3fn).view(torch.uint8)
    return codes.flatten(-2), (e + 127).to(torch.uint8)


def _pack(latent, rope, cache):
    """Rows as the pages hold them: latent fp32 [n, 512], rope fp32 [n, 64]."""
    if cache == "f16":
        return torch.cat([latent, rope], -1).half()
    codes, scales = _quantise(latent)
    return torch.cat([codes, rope.half().view(torch.uint8), scales], -1)


def _unpack(rows):
    """Rows of pages (fp16 [..., 576] or uint8 [..., 656]) as fp32 [..., 576]."""
    if rows.dtype == torch.float16:
        return rows.float()
    codes = rows[..., :LAT].contiguous().view(torch.float8_e4m3fn).float()
    scale = torch.exp2(rows[..., 640:].float() - 127.0).repeat_interleave(32, dim=-1)
    return torch.cat([codes * scale, rows[..., LAT:640].contiguous().view(torch.float16).float()], -1)


def prepare(case, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    new, length = _lengths(case)
    B, ps = case["batch"], case["page"]
    need = [-(-l // ps) for l in length]
    n_pages = sum(need) + 3
    order = torch.randperm(n_pages, generator=g, device="cuda").to(torch.int32)
    width = max(need)
    table = torch.full((B, width), -1, dtype=torch.int32, device="cuda")
    at = 0
    for b, k in enumerate(need):
        table[b, :k] = order[at:at + k]
        at += k
    rows = torch.randn(n_pages * ps, ROW, generator=g, device="cuda").bfloat16().float()
    s = {
        "case": case,
        "pages": _pack(rows[:, :LAT], rows[:, LAT:], case["cache"]).unflatten(0, (n_pages, ps)),
        "table": table,
        "cu": torch.tensor(np.concatenate([[0], np.cumsum(new)]), dtype=torch.int32, device="cuda"),
        "len": torch.tensor(length, dtype=torch.int32, device="cuda"),
    }
    T = sum(new)
    if case["kind"] == "attn":
        H = case["heads"]
        s["q_lat"] = torch.randn(T, H, LAT, generator=g, device="cuda").half()
        s["q_pe"] = torch.randn(T, H, ROPE, generator=g, device="cuda").bfloat16()
        s["out"] = torch.empty(T, H, LAT, dtype=torch.float16, device="cuda")
    else:
        back = [n + case["extra"] for n in new]
        s["c_kv"] = torch.randn(T, LAT, generator=g, device="cuda").bfloat16()
        s["k_pe"] = torch.randn(T, ROPE, generator=g, device="cuda").bfloat16()
        s["row0"] = torch.tensor([l - r for l, r in zip(length, back)], dtype=torch.int32, device="cuda")
        s["cu_rows"] = torch.tensor(np.concatenate([[0], np.cumsum(back)]), dtype=torch.int32, device="cuda")
        s["out"] = torch.empty(sum(back), ROW, dtype=torch.bfloat16, device="cuda")
    return s


def _attend_plain(s):
    case = s["case"]
    B, H, T = case["batch"], case["heads"], s["q_lat"].shape[0]
    cu, length = s["cu"].long(), s["len"].long()
    new = cu[1:] - cu[:-1]
    N = case["new_hi"]
    keys = _unpack(s["pages"][s["table"].clamp(min=0).long()]).flatten(1, 2)      # [B, K, 576]
    K = keys.shape[1]
    i = torch.arange(N, device="cuda")
    tok = (cu[:-1, None] + i).clamp(max=T - 1)                                      # [B, N]
    q = torch.cat([s["q_lat"].float(), s["q_pe"].float()], -1)[tok]                 # [B, N, H, 576]
    pos = (length - new)[:, None] + i                                               # [B, N]
    j = torch.arange(K, device="cuda")
    seen = j <= pos[..., None]                                                      # [B, N, K]
    if case["window"]:
        seen &= (j > pos[..., None] - case["window"]) | (j < case["sinks"])
    x = torch.matmul(q.flatten(1, 2), keys.transpose(1, 2)).unflatten(1, (N, H)).mul_(SCALE)
    x.masked_fill_(~seen[:, :, None], -math.inf)
    x -= x.amax(-1, keepdim=True)
    x.exp_()
    total = x.sum(-1, keepdim=True)
    o = torch.matmul(x.flatten(1, 2), keys[..., :LAT]).unflatten(1, (N, H)) / total
    t = torch.arange(T, device="cuda")
    b = torch.searchsorted(cu[1:].contiguous(), t, right=True)
    return o[b, t - cu[b]].half()


def _cache_plain(s):
    case, ps = s["case"], s["case"]["page"]
    cu, length, T = s["cu"].long(), s["len"].long(), s["c_kv"].shape[0]
    t = torch.arange(T, device="cuda")
    b = torch.searchsorted(cu[1:].contiguous(), t, right=True)
    pos = length[b] - (cu[b + 1] - t)
    # angles of far positions in 64 bits
    turn = np.float64(np.float32(FREQ_SCALE)) * np.float64(FREQ_BASE) ** (-np.arange(0, ROPE, 2) / ROPE)
    angle = pos[:, None].double() * torch.tensor(turn, device="cuda")
    cos, sin = torch.cos(angle).float(), torch.sin(angle).float()
    x = s["k_pe"].float().unflatten(-1, (ROPE // 2, 2))
    rope = torch.stack([x[..., 0] * cos - x[..., 1] * sin, x[..., 0] * sin + x[..., 1] * cos], -1).flatten(-2)
    flat = s["pages"].flatten(0, 1)
    flat[s["table"][b, pos // ps].long() * ps + pos % ps] = _pack(s["c_kv"].float(), rope, case["cache"])
    cr = s["cu_rows"].long()
    r = torch.arange(s["out"].shape[0], device="cuda")
    b = torch.searchsorted(cr[1:].contiguous(), r, right=True)
    pos = s["row0"].long()[b] + r - cr[b]
    return _unpack(flat[s["table"][b, pos // ps].long() * ps + pos % ps]).bfloat16()


def run(s):
    case = s["case"]
    if own:
        import mla_latent_kv_lat_gb300 as mla
        if case["kind"] == "attn":
            if "workspace" not in s:
                s["workspace"] = torch.empty(mla.mla_paged_workspace_size(case["heads"]), dtype=torch.uint8, device="cuda")
            mla.mla_attn_paged(s["q_lat"], s["q_pe"], s["pages"], s["table"], s["cu"], s["len"], s["out"],
                               window=case["window"], n_sink=case["sinks"], workspace=s["workspace"], scale=SCALE)
        else:
            mla.mla_paged_append(s["c_kv"], s["k_pe"], s["pages"], s["table"], s["cu"], s["len"],
                                 freq_base=FREQ_BASE, freq_scale=FREQ_SCALE)
            mla.mla_paged_gather(s["pages"], s["table"], s["row0"], s["cu_rows"], s["out"])
        return s["out"]
    return _attend_plain(s) if case["kind"] == "attn" else _cache_plain(s)


def _row_bytes(case):
    return 2 * ROW if case["cache"] == "f16" else ROW8


def _visible(case):
    """(visible pairs of a token and a key, rows that some token sees) over the batch."""
    pairs = rows = 0
    w, k = case["window"], case["sinks"]
    for n, l in zip(*_lengths(case)):
        p = np.arange(l - n, l, dtype=np.int64)
        lo = np.maximum(0, p - w + 1) if w else np.zeros_like(p)
        pairs += int((p + 1 - lo + np.minimum(k if w else 0, lo)).sum())
        rows += int(l - lo[0] + min(k if w else 0, lo[0]))
    return pairs, rows


def work(case):
    new, length = _lengths(case)
    if case["kind"] == "attn":
        pairs, rows = _visible(case)
        return {"bytes": rows * _row_bytes(case) + sum(new) * case["heads"] * (2 * ROW + 2 * LAT),
                "flops": 2 * (ROW + LAT) * pairs * case["heads"]}
    back = sum(n + case["extra"] for n in new)
    return {"bytes": sum(new) * (2 * ROW + _row_bytes(case)) + back * (_row_bytes(case) + 2 * ROW), "flops": 0}


# ---------------------------------------------------------------------------
# The definition in 64 bits, a sequence at a time.
# ---------------------------------------------------------------------------
def _e4m3_values():
    v = np.empty(256)
    for c in range(256):
        e, m = (c >> 3) & 15, c & 7
        v[c] = (m / 8 * 2.0 ** -6 if e == 0 else (1 + m / 8) * 2.0 ** (e - 7)) * (-1 if c & 128 else 1)
    v[127] = v[255] = math.nan
    return v


def _rows64(s, b, p0, p1):
    """Rows [p0, p1) of sequence b as the pages hold them, in 64 bits."""
    ps = s["case"]["page"]
    p = torch.arange(p0, p1, device="cuda")
    flat = s["pages"].flatten(0, 1)
    r = flat[s["table"][b].long()[p // ps] * ps + p % ps]
    if r.dtype == torch.float16:
        return r.double()
    lat = torch.tensor(_e4m3_values(), device="cuda")[r[:, :LAT].long()].reshape(-1, 16, 32)
    lat = lat * torch.pow(2.0, r[:, 640:].double() - 127)[..., None]
    return torch.cat([lat.reshape(-1, LAT), r[:, LAT:640].contiguous().view(torch.float16).double()], -1)


def _exact_attn(case, s):
    new, length = _lengths(case)
    if 2.0 * (ROW + LAT) * case["heads"] * sum(n * l for n, l in zip(new, length)) > 8e12:
        return None
    H, out, at = case["heads"], [], 0
    for b, (n, l) in enumerate(zip(new, length)):
        rows = _rows64(s, b, 0, l)
        step = max(1, 2 * 10 ** 8 // (l * H))
        for i0 in range(0, n, step):
            i1 = min(n, i0 + step)
            q = torch.cat([s["q_lat"][at + i0:at + i1].double(), s["q_pe"][at + i0:at + i1].double()], -1)
            x = (q.reshape(-1, ROW) @ rows.T).reshape(i1 - i0, H, l) * SCALE
            p = torch.arange(l - n + i0, l - n + i1, device="cuda")[:, None]
            j = torch.arange(l, device="cuda")
            hidden = j > p
            if case["window"]:
                hidden = hidden | ((p - j >= case["window"]) & (j >= case["sinks"]))
            x = x.masked_fill(hidden[:, None], -math.inf).softmax(-1)
            out.append((x.reshape(-1, l) @ rows[:, :LAT]).reshape(i1 - i0, H, LAT))
        at += n
    return torch.cat(out)


def _exact_cache(case, s):
    new, length = _lengths(case)
    grid = torch.tensor(sorted(v for v in set(_e4m3_values().tolist()) if v >= 0), device="cuda", dtype=torch.float64)
    out, at = [], 0
    freq = float(np.float32(FREQ_SCALE)) * float(np.float32(FREQ_BASE)) ** (-np.arange(ROPE // 2) / (ROPE // 2))
    for b, (n, l) in enumerate(zip(new, length)):
        if case["extra"]:
            out.append(_rows64(s, b, l - n - case["extra"], l - n))
        lat = s["c_kv"][at:at + n].double()
        if case["cache"] == "e4m3":
            x = lat.reshape(n, 16, 32)
            amax = x.abs().amax(-1, keepdim=True)
            d = torch.full_like(amax, 2.0 ** 7)
            for e in range(6, -16, -1):
                d = torch.where(amax <= 448 * 2.0 ** e, torch.full_like(d, 2.0 ** e), d)
            y = (x / d).abs()
            k = torch.searchsorted(grid, y.clamp(max=448)).clamp(1, len(grid) - 1)
            lo, hi = grid[k - 1], grid[k]
            # to the nearer neighbour; a tie goes to the even code, and grid is in the order of the codes
            up = (y - lo > hi - y) | ((y - lo == hi - y) & (k % 2 == 0))
            lat = (torch.where(up, hi, lo) * torch.sign(x) * d).reshape(n, LAT)
        a = torch.arange(l - n, l, device="cuda", dtype=torch.float64)[:, None] * torch.tensor(freq, device="cuda")
        x, y = s["k_pe"][at:at + n, 0::2].double(), s["k_pe"][at:at + n, 1::2].double()
        rope = torch.empty(n, ROPE, dtype=torch.float64, device="cuda")
        rope[:, 0::2] = x * torch.cos(a) - y * torch.sin(a)
        rope[:, 1::2] = x * torch.sin(a) + y * torch.cos(a)
        out.append(torch.cat([lat, rope], -1))
        at += n
    return torch.cat(out)


def exact(case, seed):
    s = prepare(case, seed)
    return _exact_attn(case, s) if case["kind"] == "attn" else _exact_cache(case, s)
