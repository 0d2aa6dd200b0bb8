"""Cases of the block-sparse paged attention and of what feeds it, in plain torch form and as the library's calls.

A case's "kind" is
  "norm"    mla_paged_norm_append: RMS norms of queries (192 values a head) and latents (512), both rotations, and the
            new rows into their pages (read back with mla_paged_gather where the pages hold 8-bit codes);
  "keys"    mla_paged_block_keys: the mean row of every block of 64 cache rows that the new tokens complete;
  "scores"  mla_paged_block_scores: scale times the largest head's product with each earlier block's mean row;
  "select"  mla_paged_select_blocks: a token's own block, the ones just before, the first ones and the best-scored;
  "attn"    mla_attn_paged_blocks: attention of each token over the rows of its listed blocks.
A batch has "batch" sequences; sequence b holds len[b] rows (len_lo..len_hi) of which the last new[b] (new_lo..new_hi)
are this call's tokens.  "cache" is the page type: "f16" (576 fp16 a row) or "e4m3" (656 bytes a row: 512 codes, 64
fp16, 16 power-of-two scales); "page" the rows of a page; "blocks" the entries of a token's list.
"""
import math
import random

import numpy as np
import torch

own = False

LAT, ROPE, NOPE, ROW, ROW8, BLOCK = 512, 64, 128, 576, 656, 64
SCALE = 1.0 / math.sqrt(192.0)
FREQ_BASE, FREQ_SCALE, EPS = 10000.0, 0.025, 1e-6


def _case(name, kind, batch, new, length, **more):
    return dict(name=name, kind=kind, batch=batch, new_lo=new[0], new_hi=new[1], len_lo=length[0], len_hi=length[1],
                **more)


def listed():
    return [
        # the projections' outputs of a serving batch's next tokens: latency
        _case("norm_tokens_b64_h128", "norm", 64, (1, 1), (1000, 65536), cache="f16", page=64, heads=128,
              q_norm=False, packed=True),
        # a long prompt's chunk into an 8-bit cache, queries normed for each head
        _case("norm_chunk_8192_h128_e4m3", "norm", 1, (8192, 8192), (40960, 40960), cache="e4m3", page=64, heads=128,
              q_norm=True, packed=False),
        # one step of a serving batch: a sequence in 64 completes a block
        _case("keys_tokens_b64_e4m3", "keys", 64, (1, 1), (1000, 65536), cache="e4m3", page=128),
        # a long prompt's rows, as it is read in
        _case("keys_prompt_98304_f16", "keys", 1, (98304, 98304), (98304, 98304), cache="f16", page=64),
        # one user's next token, 16 heads, a middling context: latency
        _case("scores_token_b1_h16", "scores", 1, (1, 1), (20001, 20001), page=64, heads=16),
        # a serving batch's next tokens, 128 heads, contexts of 4K to 98K
        _case("scores_tokens_b32_h128", "scores", 32, (1, 1), (4096, 98304), page=128, heads=128),
        # a chunk of a long prompt
        _case("scores_chunk_512_h128_at32k", "scores", 1, (512, 512), (33280, 33280), page=64, heads=128),
        # the choice for a serving batch's next tokens
        _case("select_tokens_b32", "select", 32, (1, 1), (4096, 98304), blocks=32, sinks=1, local=2),
        # the choice for chunks of several prompts
        _case("select_chunks_b3", "select", 3, (701, 2048), (20000, 65536), blocks=64, sinks=1, local=4),
        # a serving batch's next tokens over 2048 rows each
        _case("attn_tokens_b32_h128", "attn", 32, (1, 1), (4096, 98304), cache="f16", page=64, heads=128, blocks=32,
              sinks=1, local=2),
        # a chunk of a long prompt, each token over 2048 rows
        _case("attn_chunk_1024_h128_at32k", "attn", 1, (1024, 1024), (33792, 33792), cache="f16", page=64, heads=128,
              blocks=32, sinks=1, local=2),
        # ragged chunks behind an 8-bit prefix, 64 heads, odd list lengths
        _case("attn_chunks_b3_h64_e4m3", "attn", 3, (77, 301), (600, 9001), cache="e4m3", page=128, heads=64, blocks=23,
              sinks=2, local=3),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    kind = rng.choice(("norm", "keys", "scores", "select", "attn", "attn"))
    cache, page = rng.choice(("f16", "e4m3")), rng.choice((64, 128, 256))
    heads = 16 * rng.randint(1, 8)
    blocks = _log(rng, 4, 64)
    sinks, local = rng.randint(0, 2), rng.randint(1, 2)
    single = rng.random() < 0.5
    batch = _log(rng, 1, 64) if single else rng.randint(1, 4)
    if kind == "norm":
        page = rng.choice((16, 32, 64, 256))
        hi = 1 if single else _log(rng, 2, 8192 * 128 // (heads * batch))
        c = _case(None, kind, batch, (max(1, hi // 2), hi), (hi, hi + rng.randrange(0, 30000)), cache=cache, page=page,
                  heads=heads, q_norm=rng.random() < 0.5, packed=rng.random() < 0.5)
    elif kind == "keys":
        hi = 1 if single else _log(rng, 2, 98304 // batch)
        c = _case(None, kind, batch, (max(1, hi // 3), hi), (hi, hi + rng.randrange(0, 30000)), cache=cache, page=page)
    elif kind == "scores":
        hi = 1 if single else _log(rng, 2, 2048)
        length = hi + _log(rng, 1, 98304)
        length = max(hi, min(length, 512 * 128 * 33280 // (heads * batch * hi)))
        c = _case(None, kind, batch, (max(1, hi // 2), hi), (max(hi, length // 3), length), page=page, heads=heads)
    elif kind == "select":
        hi = 1 if single else _log(rng, 2, 2048)
        length = hi + _log(rng, 1, 98304)
        c = _case(None, kind, batch, (max(1, hi // 2), hi), (hi, length), blocks=max(blocks, sinks + local),
                  sinks=sinks, local=local)
    else:
        hi = 1 if single else _log(rng, 2, 1024)
        blocks = max(sinks + local, min(blocks, 1024 * 128 * 32 // (heads * batch * hi)))
        hi = max(1, min(hi, 1024 * 128 * 32 // (heads * batch * blocks)))
        length = hi + _log(rng, 1, 65536)
        c = _case(None, kind, batch, (max(1, hi // 2), hi), (max(hi, length // 3), length), cache=cache, page=page,
                  heads=heads, blocks=blocks, sinks=sinks, local=local)
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
    return new, [max(n, l) for n, l in zip(new, length)]


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
    B, T, kind = case["batch"], sum(new), case["kind"]
    s = {
        "case": case,
        "cu": torch.tensor(np.concatenate([[0], np.cumsum(new)]), dtype=torch.int32, device="cuda"),
        "len": torch.tensor(length, dtype=torch.int32, device="cuda"),
    }
    if kind != "select":
        ps = case["page"]
        need = [-(-l // ps) for l in length]
        n_pages = sum(need) + 3
        order = torch.randperm(n_pages, generator=g, device="cuda").to(torch.int32)
        table = torch.full((B, max(need)), -1, dtype=torch.int32, device="cuda")
        at = 0
        for b, k in enumerate(need):
            table[b, :k] = order[at:at + k]
            at += k
        s["table"] = table
    if kind in ("norm", "keys", "attn"):
        rows = torch.randn(n_pages * ps, ROW, generator=g, device="cuda").bfloat16().float()
        s["pages"] = _pack(rows[:, :LAT], rows[:, LAT:], case["cache"]).unflatten(0, (n_pages, ps))
        del rows
    if kind in ("keys", "scores"):
        # means of 64 rows
        s["keys"] = (torch.randn(n_pages, ps // BLOCK, ROW, generator=g, device="cuda") * 0.125).half()
    if kind in ("scores", "attn"):
        H = case["heads"]
        s["q_lat"] = torch.randn(T, H, LAT, generator=g, device="cuda").half()
        s["q_pe"] = torch.randn(T, H, ROPE, generator=g, device="cuda").bfloat16()
    if kind == "norm":
        H = case["heads"]
        if case["packed"]:                  # both projections' outputs side by side in one buffer
            both = torch.randn(T, H * (NOPE + ROPE) + ROW, generator=g, device="cuda").bfloat16()
            s["q"] = both[:, :H * (NOPE + ROPE)].unflatten(1, (H, NOPE + ROPE))
            s["kv"] = both[:, H * (NOPE + ROPE):]
        else:
            s["q"] = torch.randn(T, H, NOPE + ROPE, generator=g, device="cuda").bfloat16()
            s["kv"] = torch.randn(T, ROW, generator=g, device="cuda").bfloat16()
        s["q_weight"] = (1 + 0.25 * torch.randn(NOPE + ROPE, generator=g, device="cuda")).bfloat16() if case["q_norm"] else None
        s["kv_weight"] = (1 + 0.25 * torch.randn(LAT, generator=g, device="cuda")).bfloat16()
        s["q_nope"] = torch.empty(T, H, NOPE, dtype=torch.bfloat16, device="cuda")
        s["q_pe"] = torch.empty(T, H, ROPE, dtype=torch.bfloat16, device="cuda")
        if case["cache"] == "e4m3":
            s["row0"] = s["len"] - torch.diff(s["cu"])
            s["rows"] = torch.empty(T, ROW, dtype=torch.float16, device="cuda")
    wide = max(-(-l // BLOCK) for l in length)
    if kind in ("scores", "select"):
        s["scores"] = torch.randn(T, wide, generator=g, device="cuda") if kind == "select" else torch.empty(T, wide, device="cuda")
    if kind in ("select", "attn"):
        K = case["blocks"]
        s["blocks"] = torch.empty(T, K, dtype=torch.int32, device="cuda")
        s["counts"] = torch.empty(T, dtype=torch.int32, device="cuda")
    if kind == "attn":
        # neighbouring tokens prefer the same blocks
        like = torch.randn(B, wide, generator=g, device="cuda")[_seq_of(s)]
        s["blocks"], s["counts"] = _choose(s, like + 0.5 * torch.randn(T, wide, generator=g, device="cuda"))
        s["o"] = torch.empty(T, H, LAT, dtype=torch.float16, device="cuda")
    return s


def _seq_of(s):
    """The sequence of each token."""
    cu = s["cu"].long()
    return torch.searchsorted(cu[1:].contiguous(), torch.arange(_tokens(s), device="cuda"), right=True)


def _tokens(s):
    return sum(_lengths(s["case"])[0])


def _positions(s):
    """(sequence, position) of each token."""
    b = _seq_of(s)
    cu = s["cu"].long()
    return b, s["len"].long()[b] - (cu[b + 1] - torch.arange(b.shape[0], device="cuda"))


def _choose(s, scores):
    """(blocks [T, K], counts [T]) from scores [T, W]."""
    case = s["case"]
    K, W = case["blocks"], scores.shape[1]
    last = (_positions(s)[1] // BLOCK)[:, None]
    j = torch.arange(W, device="cuda")
    x = scores.masked_fill((j < case["sinks"]) | (j > last - case["local"]), math.inf).masked_fill(j > last, -math.inf)
    # a stable sort: equal scores stay in the order of their blocks
    order = torch.sort(x, dim=1, descending=True, stable=True).indices[:, :K]
    order = torch.where(order <= last, order, W).sort(1).values
    count = (order < W).sum(1)
    out = torch.full((scores.shape[0], K), -1, dtype=torch.int32, device="cuda")
    out[:, :order.shape[1]] = torch.where(order < W, order, -1).int()
    return out, count.int()


def _rotate(x, pos):
    """x fp32 [T, ..., 64] turned by its token's position, pairs (2i, 2i + 1); angles of far positions in 64 bits."""
    turn = np.float64(np.float32(FREQ_SCALE)) * np.float64(FREQ_BASE) ** (-np.arange(0, ROPE, 2) / ROPE)
    angle = pos[:, None].double() * torch.tensor(turn, device="cuda")
    angle = angle.view(angle.shape[0], *([1] * (x.dim() - 2)), ROPE // 2)
    cos, sin = torch.cos(angle).float(), torch.sin(angle).float()
    x = x.unflatten(-1, (ROPE // 2, 2))
    return torch.stack([x[..., 0] * cos - x[..., 1] * sin, x[..., 0] * sin + x[..., 1] * cos], -1).flatten(-2)


def _rms(x, weight):
    return x * torch.rsqrt(x.square().mean(-1, keepdim=True) + EPS) * weight.float()


def _norm_plain(s):
    case, ps = s["case"], s["case"]["page"]
    b, pos = _positions(s)
    q, kv = s["q"].float(), s["kv"].float()
    if case["q_norm"]:
        q = _rms(q, s["q_weight"])
    out = [q[..., :NOPE].bfloat16(), _rotate(q[..., NOPE:], pos).bfloat16()]
    rows = _pack(_rms(kv[:, :LAT], s["kv_weight"]), _rotate(kv[:, LAT:], pos), case["cache"])
    flat = s["pages"].flatten(0, 1)
    at = s["table"][b, pos // ps].long() * ps + pos % ps
    flat[at] = rows
    return out + [s["pages"] if case["cache"] == "f16" else _unpack(flat[at]).half()]


def _keys_plain(s):
    case, ps = s["case"], s["case"]["page"]
    b, pos = _positions(s)
    at = s["table"][b, pos // ps].long() * ps + pos % ps
    done = at[pos % BLOCK == BLOCK - 1] // BLOCK           # the pool's block that each such token completes
    rows = _unpack(s["pages"].flatten(0, 1).unflatten(0, (-1, BLOCK))[done])
    s["keys"].flatten(0, 1)[done] = rows.mean(1).half()
    return s["keys"]


def _padded(s):
    """(token index [B, N], position [B, N]) of a batch as a rectangle."""
    cu, length = s["cu"].long(), s["len"].long()
    i = torch.arange(s["case"]["new_hi"], device="cuda")
    return (cu[:-1, None] + i).clamp(max=_tokens(s) - 1), (length - cu[1:] + cu[:-1])[:, None] + i


def _scores_plain(s):
    case, (T, W) = s["case"], s["scores"].shape
    per = case["page"] // BLOCK
    j = torch.arange(W, device="cuda")
    keys = s["keys"][s["table"].clamp(min=0).long()].flatten(1, 2)[:, :W].float()       # [B, W', 576]
    tok, _ = _padded(s)
    q = torch.cat([s["q_lat"].float(), s["q_pe"].float()], -1)[tok]                      # [B, N, H, 576]
    x = torch.matmul(q.flatten(1, 2), keys.transpose(1, 2)).unflatten(1, (case["new_hi"], case["heads"])).amax(2) * SCALE
    b, pos = _positions(s)
    x = x[b, torch.arange(T, device="cuda") - s["cu"].long()[b]]
    return x.masked_fill(j >= (pos // BLOCK)[:, None], -math.inf)


def _attn_plain(s):
    case, ps = s["case"], s["case"]["page"]
    b, pos = _positions(s)
    listed_ = s["blocks"].long()
    key = (listed_.clamp(min=0)[..., None] * BLOCK + torch.arange(BLOCK, device="cuda")).flatten(1)     # [T, K * 64]
    seen = (listed_ >= 0).repeat_interleave(BLOCK, dim=1) & (key <= pos[:, None])
    page = (key // ps).clamp(max=s["table"].shape[1] - 1)
    rows = _unpack(s["pages"].flatten(0, 1)[s["table"][b[:, None], page].clamp(min=0).long() * ps + key % ps])
    q = torch.cat([s["q_lat"].float(), s["q_pe"].float()], -1)
    x = torch.matmul(q, rows.transpose(1, 2)).mul_(SCALE)
    x.masked_fill_(~seen[:, None], -math.inf)
    x -= x.amax(-1, keepdim=True)
    x.exp_()
    total = x.sum(-1, keepdim=True)
    return (torch.matmul(x, rows[..., :LAT]) / total).half()


def run(s):
    case = s["case"]
    kind = case["kind"]
    if own:
        import mla_latent_kv_lat_gb300 as mla
        if kind == "norm":
            mla.mla_paged_norm_append(s["q"], s["kv"], s["q_weight"], s["kv_weight"], s["pages"], s["table"], s["cu"],
                                      s["len"], s["q_nope"], s["q_pe"], eps=EPS, freq_base=FREQ_BASE, freq_scale=FREQ_SCALE)
            if case["cache"] == "f16":
                return [s["q_nope"], s["q_pe"], s["pages"]]
            mla.mla_paged_gather(s["pages"], s["table"], s["row0"], s["cu"], s["rows"])
            return [s["q_nope"], s["q_pe"], s["rows"]]
        if kind == "keys":
            if "T" not in s:                # a program knows how many tokens its batch has
                s["T"] = _tokens(s)
            mla.mla_paged_block_keys(s["pages"], s["table"], s["cu"], s["len"], s["keys"], s["T"])
            return s["keys"]
        if kind == "scores":
            mla.mla_paged_block_scores(s["q_lat"], s["q_pe"], s["keys"], s["table"], s["cu"], s["len"], s["scores"], scale=SCALE)
            return s["scores"]
        if kind == "select":
            mla.mla_paged_select_blocks(s["scores"], s["cu"], s["len"], s["blocks"], s["counts"], n_sink=case["sinks"],
                                        n_local=case["local"])
            return [s["blocks"], s["counts"]]
        if "workspace" not in s:
            s["workspace"] = torch.empty(mla.mla_paged_workspace_size(case["heads"]), dtype=torch.uint8, device="cuda")
        mla.mla_attn_paged_blocks(s["q_lat"], s["q_pe"], s["pages"], s["table"], s["cu"], s["len"], s["blocks"], s["counts"],
                                  s["o"], workspace=s["workspace"], scale=SCALE)
        return s["o"]
    if kind == "select":
        return list(_choose(s, s["scores"]))
    return {"norm": _norm_plain, "keys": _keys_plain, "scores": _scores_plain, "attn": _attn_plain}[kind](s)


def _row_bytes(case):
    return 2 * ROW if case["cache"] == "f16" else ROW8


def work(case):
    new, length = _lengths(case)
    kind, T = case["kind"], sum(new)
    if kind == "norm":
        qkv = 2 * T * (case["heads"] * (NOPE + ROPE) * 2 + ROW)
        back = 0 if case["cache"] == "f16" else T * (ROW8 + 2 * ROW)
        return {"bytes": qkv + T * _row_bytes(case) + back, "flops": 0}
    if kind == "keys":
        done = sum(l // BLOCK - (l - n) // BLOCK for n, l in zip(new, length))
        return {"bytes": done * (BLOCK * _row_bytes(case) + 2 * ROW) + 8 * len(new), "flops": 0}
    wide = max(-(-l // BLOCK) for l in length)
    if kind == "scores":
        pairs = sum(int((np.arange(l - n, l) // BLOCK).sum()) for n, l in zip(new, length))
        keys = sum((l - 1) // BLOCK for l in length)
        return {"bytes": T * case["heads"] * 2 * ROW + keys * 2 * ROW + 4 * T * wide, "flops": 2 * ROW * pairs * case["heads"]}
    if kind == "select":
        pairs = sum(int((np.arange(l - n, l) // BLOCK).sum()) for n, l in zip(new, length))
        return {"bytes": 4 * pairs + 4 * T * (case["blocks"] + 1), "flops": 0}
    entries = rows = 0
    for n, l in zip(new, length):
        k = np.minimum(np.arange(l - n, l) // BLOCK + 1, case["blocks"])
        entries += int(k.sum())
        rows += min(l, int(k.sum()) * BLOCK)
    return {"bytes": rows * _row_bytes(case) + T * case["heads"] * (2 * ROW + 2 * LAT) + 4 * T * (case["blocks"] + 1),
            "flops": 2 * (ROW + LAT) * entries * BLOCK * case["heads"]}


# ---------------------------------------------------------------------------
# The definitions in 64 bits, a sequence at a time.
# ---------------------------------------------------------------------------
def _e4m3_values():
    v = np.empty(256)
    for c in range(256):
        e, m = (c >> 3) & 15, c & 7
        v[c] = (m / 8 * 2.0 ** -6 if e == 0 else (1 + m / 8) * 2.0 ** (e - 7)) * (-1 if c & 128 else 1)
    v[127] = v[255] = math.nan
    return v


def _values64(s, r):
    """Raw rows of pages in 64 bits."""
    if r.dtype == torch.float16:
        return r.double()
    lat = torch.tensor(_e4m3_values(), device="cuda")[r[..., :LAT].long()].unflatten(-1, (16, 32))
    lat = lat * torch.pow(2.0, r[..., 640:].double() - 127)[..., None]
    return torch.cat([lat.flatten(-2), r[..., LAT:640].contiguous().view(torch.float16).double()], -1)


def _rows64(s, b, p0, p1):
    """Rows [p0, p1) of sequence b as the pages hold them, in 64 bits."""
    ps = s["case"]["page"]
    p = torch.arange(p0, p1, device="cuda")
    return _values64(s, s["pages"].flatten(0, 1)[s["table"][b].long()[p // ps] * ps + p % ps])


def _e4m3_64(lat):
    """Latents in 64 bits [n, 512] -> the values that their e4m3 codes and scales stand for."""
    grid = torch.tensor(sorted(v for v in set(_e4m3_values().tolist()) if v >= 0), device="cuda", dtype=torch.float64)
    x = lat.reshape(-1, 16, 32)
    amax = x.abs().amax(-1, keepdim=True)
    d = torch.full_like(amax, 2.0 ** 7)
    for e in range(6, -16, -1):
        d = torch.where(amax <= 448 * 2.0 ** e, torch.full_like(d, 2.0 ** e), d)
    y = (x / d).abs()
    k = torch.searchsorted(grid, y.clamp(max=448)).clamp(1, len(grid) - 1)
    lo, hi = grid[k - 1], grid[k]
    # to the nearer neighbour; a tie goes to the even code, and grid is in the order of the codes
    up = (y - lo > hi - y) | ((y - lo == hi - y) & (k % 2 == 0))
    return (torch.where(up, hi, lo) * torch.sign(x) * d).reshape(-1, LAT)


def _exact_norm(case, s):
    new, length = _lengths(case)
    ps = case["page"]
    freq = torch.tensor(float(np.float32(FREQ_SCALE)) * float(np.float32(FREQ_BASE)) ** (-np.arange(ROPE // 2) / (ROPE // 2)), device="cuda")
    pages = s["pages"].double() if case["cache"] == "f16" else None
    nope, pe, out, at = [], [], [], 0
    for b, (n, l) in enumerate(zip(new, length)):
        for i0 in range(0, n, 1024):
            i1 = min(n, i0 + 1024)
            p = torch.arange(l - n + i0, l - n + i1, device="cuda")
            a = p.double()[:, None] * freq

            def turn(x, a):
                u, v = x[..., 0::2], x[..., 1::2]
                y = torch.empty_like(x)
                y[..., 0::2] = u * torch.cos(a) - v * torch.sin(a)
                y[..., 1::2] = u * torch.sin(a) + v * torch.cos(a)
                return y

            q = s["q"][at + i0:at + i1].double()
            if case["q_norm"]:
                q = q / torch.sqrt((q * q).sum(-1, keepdim=True) / (NOPE + ROPE) + EPS) * s["q_weight"].double()
            nope.append(q[..., :NOPE].clone())
            pe.append(turn(q[..., NOPE:], a[:, None]))
            kv = s["kv"][at + i0:at + i1].double()
            lat = kv[:, :LAT] / torch.sqrt((kv[:, :LAT] ** 2).sum(-1, keepdim=True) / LAT + EPS) * s["kv_weight"].double()
            rope = turn(kv[:, LAT:], a)
            if pages is None:
                out.append(torch.cat([_e4m3_64(lat), rope], -1))
            else:
                pages.flatten(0, 1)[s["table"][b].long()[p // ps] * ps + p % ps] = torch.cat([lat, rope], -1)
        at += n
    return [torch.cat(nope), torch.cat(pe), torch.cat(out) if pages is None else pages]


def _exact_keys(case, s):
    new, length = _lengths(case)
    ps, keys = case["page"], s["keys"].double()
    for b, (n, l) in enumerate(zip(new, length)):
        for j0 in range((l - n) // BLOCK, l // BLOCK, 128):
            j = torch.arange(j0, min(j0 + 128, l // BLOCK), device="cuda")
            m = _rows64(s, b, j0 * BLOCK, (j0 + len(j)) * BLOCK).reshape(-1, BLOCK, ROW).sum(1) / BLOCK
            keys[s["table"][b].long()[j * BLOCK // ps], j % (ps // BLOCK)] = m
    return keys


def _exact_scores(case, s):
    new, length = _lengths(case)
    if 2.0 * ROW * case["heads"] / BLOCK * sum(n * l for n, l in zip(new, length)) > 4e12:
        return None
    H, per, at = case["heads"], case["page"] // BLOCK, 0
    out = torch.full(tuple(s["scores"].shape), -math.inf, dtype=torch.float64, device="cuda")
    for b, (n, l) in enumerate(zip(new, length)):
        m = (l - 1) // BLOCK
        if m:
            j = torch.arange(m, device="cuda")
            k = s["keys"][s["table"][b].long()[j // per], j % per].double()
            step = max(1, 10 ** 8 // (m * H))
            for i0 in range(0, n, step):
                i1 = min(n, i0 + step)
                q = torch.cat([s["q_lat"][at + i0:at + i1].double(), s["q_pe"][at + i0:at + i1].double()], -1)
                x = (q.reshape(-1, ROW) @ k.T).reshape(i1 - i0, H, m).max(1).values * SCALE
                p = torch.arange(l - n + i0, l - n + i1, device="cuda")[:, None]
                out[at + i0:at + i1, :m] = torch.where(j < p // BLOCK, x, torch.full_like(x, -math.inf))
        at += n
    return out


def _exact_attn(case, s):
    new, length = _lengths(case)
    if work(case)["flops"] > 4e12:
        return None
    H, K, out, at = case["heads"], case["blocks"], [], 0
    for b, (n, l) in enumerate(zip(new, length)):
        rows = _rows64(s, b, 0, l)
        step = max(1, 10 ** 8 // (K * BLOCK * ROW))
        for i0 in range(0, n, step):
            i1 = min(n, i0 + step)
            t = s["blocks"][at + i0:at + i1].long()
            p = torch.arange(l - n + i0, l - n + i1, device="cuda")
            key = (t * BLOCK)[..., None] + torch.arange(BLOCK, device="cuda")
            hidden = ((t < 0)[..., None] | (key > p[:, None, None])).reshape(i1 - i0, 1, -1)
            r = rows[key.clamp(min=0, max=l - 1).reshape(i1 - i0, -1)]
            q = torch.cat([s["q_lat"][at + i0:at + i1].double(), s["q_pe"][at + i0:at + i1].double()], -1)
            w = (q @ r.transpose(1, 2) * SCALE).masked_fill(hidden, -math.inf).softmax(-1)
            out.append(w @ r[..., :LAT])
        at += n
    return torch.cat(out)


def exact(case, seed):
    if case["kind"] == "select":
        return None
    s = prepare(case, seed)
    return {"norm": _exact_norm, "keys": _exact_keys, "scores": _exact_scores, "attn": _exact_attn}[case["kind"]](case, s)
