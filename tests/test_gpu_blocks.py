"""Normed appends, mean rows, block scores, the choice of blocks and attention over listed blocks on the GPU, against
the 64-bit definitions, with bounds per value that follow from the arithmetic."""
import numpy as np
import pytest
import torch

import mla_latent_kv_lat_gb300 as mla
from oracle import blocks_oracle as BO
from oracle import mla_oracle as O
from oracle import paged_oracle as PO
from tests.paged_util import SCALE, Batch, bf16

pytestmark = pytest.mark.gpu

INVALID, RANGE = -1, -7
FB, FS, EPS = float(np.float32(10000.0)), float(np.float32(0.025)), float(np.float32(1e-6))
BATCHES = [(64, [1], [1], 0), (64, [1], [64], 0), (64, [1, 0, 3, 1], [700, 0, 3, 64], 2),
           (128, [130, 65, 1], [131, 1000, 129], 0), (256, [255, 300], [5000, 300], 5), (4096, [1, 70], [4097, 8000], 1)]


@pytest.fixture(scope="module", autouse=True)
def _lib():
    if not torch.cuda.is_available():
        pytest.skip("needs a CUDA device")
    from mla_latent_kv_lat_gb300 import build
    build.build()
    mla.load_library()
    assert mla.mla_get_device_error() == 0


def i32(x):
    return torch.tensor(np.asarray(x, np.int32), device="cuda")


def host(t):
    return t.double().cpu().numpy()


def positions(b):
    return np.concatenate([np.arange(l - n, l) for n, l in zip(b.news, b.lens)] + [np.zeros(0, int)])


def full_table(b):
    """The batch's table with every page of a sequence in it."""
    table = b.table.copy()
    for s in range(b.B):
        p = np.arange(0, b.lens[s], b.ps)
        table[s, :len(p)] = b.row_ids[s][p] // b.ps
    return torch.from_numpy(table).cuda()


# ---------------------------------------------------------------------------
# norms, rotation, append
# ---------------------------------------------------------------------------
def rel_norm(n):
    """How far a normed value may be off before its last rounding, relative: the fp32 sum of n squares (all positive;
    at most n / 8 + 8 roundings deep) halved by the root, the reciprocal root (2^-22), two products (2^-24 each)."""
    return (n / 8 + 8) / 2 * 2.0 ** -24 + 2.0 ** -22 + 2.0 ** -23


def check_rotated(got, x, pos, half_step, rel):
    """got against the rotation of x [.., 64] (64 bits) at pos: off by rel and by sine, cosine and the rotation in fp32
    (a few 2^-24 of the pair's length), then by half a step."""
    want = PO.rope_rows(x, pos, FB, FS)
    pair = np.repeat(np.hypot(x[..., 0::2], x[..., 1::2]), 2, axis=-1)
    assert (np.abs(got - want) <= half_step * np.abs(want) + (rel + 1e-6) * pair + 2.0 ** -25).all()


@pytest.mark.parametrize("e4m3", [False, True])
@pytest.mark.parametrize("H,q_norm,packed", [(16, True, True), (48, False, False), (128, True, False)])
@pytest.mark.parametrize("ps,news,lens,pad", [(16, [1], [1], 0)] + BATCHES[2:5])
def test_norm_append(e4m3, H, q_norm, packed, ps, news, lens, pad):
    b = Batch(5, e4m3, 16, ps, news, lens, pad=pad)
    rng = np.random.default_rng(6)
    q = bf16(rng.standard_normal((b.T, H, 192)) * np.exp(rng.uniform(-6, 6, (b.T, H, 1))))
    kv = bf16(rng.standard_normal((b.T, 576)) * np.exp(rng.uniform(-6, 6, (b.T, 1))))
    q[0, 0], kv[0, :512] = 0.0, 0.0                       # nothing to norm
    kv[-1 - pad, :100] *= 2.0 ** -30                      # blocks of tiny values
    qw, kw = bf16(1 + 0.3 * rng.standard_normal(192)), bf16(1 + 0.3 * rng.standard_normal(512))
    n = int(b.cu[-1])
    q[n:], kv[n:] = np.nan, np.nan
    dq, dkv = torch.from_numpy(q).bfloat16().cuda(), torch.from_numpy(kv).bfloat16().cuda()
    if packed:                                            # slices of one wider buffer
        both = torch.full((b.T, H * 192 + 576 + 24), 7.0, dtype=torch.bfloat16, device="cuda")
        both[:, 8:8 + H * 192], both[:, 8 + H * 192:584 + H * 192] = dq.flatten(1), dkv
        dq, dkv = both[:, 8:8 + H * 192].unflatten(1, (H, 192)), both[:, 8 + H * 192:584 + H * 192]
        assert b.T == 1 or not dq.is_contiguous()
    pages, table = b.pages_dev(), full_table(b)
    q_nope = torch.full((b.T, H, 128), 7.0, dtype=torch.bfloat16, device="cuda")
    q_pe = torch.full((b.T, H, 64), 7.0, dtype=torch.bfloat16, device="cuda")
    mla.mla_paged_norm_append(dq, dkv, torch.from_numpy(qw).bfloat16().cuda() if q_norm else None,
                              torch.from_numpy(kw).bfloat16().cuda(), pages, table, i32(b.cu), i32(b.lens), q_nope, q_pe,
                              eps=EPS, freq_base=FB, freq_scale=FS)
    torch.cuda.synchronize()
    assert mla.mla_get_device_error() == 0
    assert (q_nope[n:] == 7).all() and (q_pe[n:] == 7).all()
    pos = positions(b)
    x, rel = BO.rms(q[:n], qw.astype(np.float64) if q_norm else None, EPS), rel_norm(192) if q_norm else 0.0
    got = host(q_nope[:n])
    assert (np.abs(got - x[..., :128]) <= (2.0 ** -8 + 2 * rel) * np.abs(x[..., :128])).all()
    got = host(q_pe[:n])
    for h in range(0, H, 7):
        check_rotated(got[:, h], x[:, h, 128:], pos, 2.0 ** -8, 2 * rel)
    # the rows; no other byte of the pool is touched
    raw = pages.view(torch.uint8).reshape(b.raw.shape).cpu().numpy()
    slot = np.concatenate([b.row_ids[s][b.lens[s] - b.news[s]:] for s in range(b.B)]).astype(int)
    untouched = np.ones(raw.shape[0], bool)
    untouched[slot] = False
    assert np.array_equal(raw[untouched], b.raw[untouched])
    vals = PO.row_values(raw[slot], e4m3)
    lat, rel = BO.rms(kv[:n, :512], kw.astype(np.float64), EPS), 2 * rel_norm(512)
    check_rotated(vals[:, 512:], kv[:n, 512:].astype(np.float64), pos, 2.0 ** -11, 0.0)
    if not e4m3:
        assert (np.abs(vals[:, :512] - lat) <= (2.0 ** -11 + rel) * np.abs(lat) + 2.0 ** -25).all()
        return
    s = 2.0 ** (raw[slot][:, 640:].astype(np.float64) - 127)            # each 32 values' scale
    amax = np.abs(lat).reshape(n, 16, 32).max(-1)
    # the smallest scale that holds the largest value, which is known to within rel
    assert ((amax * (1 - rel) <= 448 * s) & ((amax * (1 + rel) > 224 * s) | (s == 2.0 ** -15))).all()
    s = np.repeat(s, 32, axis=1)
    # half a step of a code: 2^-4 of the value, or half the smallest step (2^-9 of the scale)
    assert (np.abs(vals[:, :512] - lat) <= (2.0 ** -4 + 2 * rel) * np.abs(lat) + 2.0 ** -10 * s).all()


def test_norm_append_takes_broadcast_inputs_and_refuses_odd_places():
    b = Batch(39, False, 16, 64, [5, 2], [70, 2])
    H, T = 32, 7
    one_q, one_kv = torch.randn(1, 1, 192, device="cuda").bfloat16(), torch.randn(1, 576, device="cuda").bfloat16()
    w, qw = torch.ones(512, dtype=torch.bfloat16, device="cuda"), torch.ones(192, dtype=torch.bfloat16, device="cuda")

    def go(q, kv):
        pages = b.pages_dev().nan_to_num_(0.0)
        outs = [torch.empty(T, H, n, dtype=torch.bfloat16, device="cuda") for n in (128, 64)]
        mla.mla_paged_norm_append(q, kv, qw, w, pages, full_table(b), i32(b.cu), i32(b.lens), *outs)
        torch.cuda.synchronize()
        assert mla.mla_get_device_error() == 0
        return outs + [pages]

    q, kv = one_q.expand(T, H, 192), one_kv.expand(T, 576)               # strides of zero
    for x, y in zip(go(q, kv), go(q.contiguous(), kv.contiguous())):
        assert torch.equal(x, y)
    heads_first = q.transpose(0, 1).contiguous().transpose(0, 1)          # [H, T, 192] in memory
    assert torch.equal(go(heads_first, kv)[1], go(q, kv)[1])
    odd = torch.zeros(T, 576 + 8, dtype=torch.bfloat16, device="cuda")
    for bad in (odd[:, 4:580], torch.zeros(T, 580, dtype=torch.bfloat16, device="cuda")[:, :576]):
        with pytest.raises(mla.MLAError) as e:
            go(q, bad)
        assert e.value.status == -3
    with pytest.raises(ValueError, match="last dimension"):
        go(q, torch.zeros(576, T, dtype=torch.bfloat16, device="cuda").t())


def test_norm_append_reports_what_rows_cannot_hold_and_bad_pages():
    b = Batch(7, False, 16, 64, [2, 1], [80, 5])
    H, n = 16, 3
    q = torch.zeros(n, H, 192, dtype=torch.bfloat16, device="cuda")
    kv = torch.ones(n, 576, dtype=torch.bfloat16, device="cuda")
    w = torch.ones(512, dtype=torch.bfloat16, device="cuda")
    outs = [torch.full((n, H, d), 7.0, dtype=torch.bfloat16, device="cuda") for d in (128, 64)]
    pages, table = b.pages_dev(), full_table(b)

    def go(kv, w, table):
        mla.mla_paged_norm_append(q, kv, None, w, pages, table, i32(b.cu), i32(b.lens), *outs)
        torch.cuda.synchronize()
        return mla.mla_get_device_error()

    assert go(kv, w, table) == 0
    assert go(kv, w * 1e5, table) == RANGE                # latents past fp16
    far = kv.clone()
    far[2, 512:] = 1e30                                   # RoPE values past fp16
    assert go(far, w, table) == RANGE
    far[2, 512:] = float("nan")
    assert go(far, w, table) == RANGE
    assert go(kv, w, table) == 0
    for o in outs:
        o.fill_(7.0)
    bad = table.clone()
    bad[0, 1] = b.n_pages                                 # the page of sequence 0's two new tokens
    before = pages.clone()
    assert go(kv, w, bad) == INVALID
    assert (outs[0] == 0).all() and (outs[1] == 0).all()  # the queries are there
    same = (pages == before).flatten(0, 1).all(-1) | before.isnan().flatten(0, 1).all(-1)
    assert same.all()                                     # (sequence 1's row is what it was: the same values again)


@pytest.mark.parametrize("e4m3", [False, True])
@pytest.mark.parametrize("H,per,q_norm", [(16, 3, True), (80, 3, True), (80, 2, False), (128, 8, True)])
def test_norm_append_of_many_tokens(e4m3, H, per, q_norm):
    """Enough tokens that a warp takes ``per`` groups of four heads (and the last one of a token what is left): the bits
    of calls with few tokens, each token's in a sample near the definition."""
    sms = torch.cuda.get_device_properties(0).multi_processor_count
    n = -(-per * 64 * sms * 4 // H)
    news = [n // 2, 3, n - n // 2]
    b = Batch(42, e4m3, 16, 64, news, [n // 2, 700, n + 100], pad=1)
    n, g = int(b.cu[-1]), torch.Generator(device="cuda").manual_seed(42)
    rnd = lambda *s: torch.randn(*s, generator=g, device="cuda")  # noqa: E731
    q, kv = (rnd(b.T, H, 192) * torch.exp(2 * rnd(b.T, H, 1))).bfloat16(), (rnd(b.T, 576) * torch.exp(2 * rnd(b.T, 1))).bfloat16()
    qw, kw = (1 + 0.3 * rnd(192)).bfloat16() if q_norm else None, (1 + 0.3 * rnd(512)).bfloat16()
    table = full_table(b)

    def go(q, kv, pages, cu, lens):
        outs = [torch.full((len(q), H, d), 7.0, dtype=torch.bfloat16, device="cuda") for d in (128, 64)]
        mla.mla_paged_norm_append(q, kv, qw, kw, pages, table, i32(cu), i32(lens), *outs, eps=EPS, freq_base=FB, freq_scale=FS)
        torch.cuda.synchronize()
        assert mla.mla_get_device_error() == 0
        return outs

    pages = [b.pages_dev().view(torch.uint8).fill_(0).view(torch.uint8 if e4m3 else torch.float16) for _ in range(2)]
    nope, pe = go(q, kv, pages[0], b.cu, b.lens)
    assert (nope[n:] == 7).all() and (pe[n:] == 7).all()
    few = 32 * sms // H                                   # half of what makes a warp take one group more
    for lo in range(0, n, few):
        hi = min(lo + few, n)
        part = np.clip(b.cu, lo, hi)
        lens = [l - n_new + int(np.clip(hi - c, 0, n_new)) for l, n_new, c in zip(b.lens, b.news, b.cu)]
        x, y = go(q[lo:hi], kv[lo:hi], pages[1], part - lo, lens)
        assert torch.equal(x, nope[lo:hi]) and torch.equal(y, pe[lo:hi]), lo
    assert torch.equal(pages[0].view(torch.uint8), pages[1].view(torch.uint8))
    some = np.unique(np.concatenate([np.arange(0, n, 41), [n - 1]]))
    pos, at = positions(b)[some], torch.from_numpy(some).cuda()
    rel = rel_norm(192) if q_norm else 0.0
    x = BO.rms(host(q[at]), host(qw) if q_norm else None, EPS)
    assert (np.abs(host(nope[at]) - x[..., :128]) <= (2.0 ** -8 + 2 * rel) * np.abs(x[..., :128])).all()
    for h in range(H):
        check_rotated(host(pe[at, h]), x[:, h, 128:], pos, 2.0 ** -8, 2 * rel)


# ---------------------------------------------------------------------------
# mean rows
# ---------------------------------------------------------------------------
@pytest.mark.parametrize("e4m3", [False, True])
@pytest.mark.parametrize("ps,news,lens,pad", BATCHES + [(64, [1] * 70, list(range(60, 130)), 0), (128, [3000], [3001], 3)])
def test_block_keys(e4m3, ps, news, lens, pad):
    b = Batch(8, e4m3, 16, ps, news, lens)
    keys = torch.full((b.n_pages, ps // 64, 576), 7.0, dtype=torch.float16, device="cuda")
    want, tol = np.full((b.n_pages * ps // 64, 576), 7.0), np.zeros((b.n_pages * ps // 64, 576))
    for s in range(b.B):
        for j in range((b.lens[s] - b.news[s]) // 64, b.lens[s] // 64):
            rows = b.rows[s][64 * j:64 * j + 64]
            at = int(b.row_ids[s][64 * j]) // 64
            want[at] = rows.mean(0)
            # 64 fp32 additions of at most sum |x|, over 64; one rounding to fp16
            tol[at] = 64 * 2.0 ** -24 * np.abs(rows).mean(0) + 2.0 ** -11 * np.abs(want[at]) + 2.0 ** -25
    mla.mla_paged_block_keys(b.pages_dev(), full_table(b), i32(b.cu), i32(b.lens), keys, b.T + pad)
    torch.cuda.synchronize()
    assert mla.mla_get_device_error() == 0
    assert (np.abs(host(keys).reshape(want.shape) - want) <= tol).all()


@pytest.mark.parametrize("e4m3", [False, True])
def test_block_keys_of_more_blocks_than_the_grid(e4m3):
    """More completed blocks than blocks of threads, 16 an SM, so that these take several."""
    ps, sms = 128, torch.cuda.get_device_properties(0).multi_processor_count
    g = torch.Generator(device="cuda").manual_seed(43)
    news, lens = [64 * 25 * sms + 10, 0, 64 * 17 * sms, 1], [64 * 25 * sms + 10, 500, 64 * 17 * sms + 700, 640]
    width = -(-max(lens) // ps)
    n_pages = sum(-(-l // ps) for l in lens) + 1
    order, table, at = np.random.default_rng(43).permutation(n_pages), np.full((4, width), -1, np.int32), 0
    for s, l in enumerate(lens):
        table[s, :-(-l // ps)] = order[at:at + -(-l // ps)]
        at += -(-l // ps)
    table, pages = i32(table), mla.paged_pages(n_pages, ps, e4m3)
    cu = np.concatenate([[0], np.cumsum(lens)])
    c_kv, k_pe = (torch.randn(int(cu[-1]), d, generator=g, device="cuda").bfloat16() for d in (512, 64))
    mla.mla_paged_append(c_kv, k_pe, pages, table, i32(cu), i32(lens))
    rows = torch.empty(int(cu[-1]), 576, dtype=torch.float16, device="cuda")
    mla.mla_paged_gather(pages, table, None, i32(cu), rows)           # (exact)
    keys = torch.full((n_pages, ps // 64, 576), 7.0, dtype=torch.float16, device="cuda")
    new = np.concatenate([[0], np.cumsum(news)])
    assert int(new[-1]) // 64 + 4 > 2 * 16 * sms
    mla.mla_paged_block_keys(pages, table, i32(new), i32(lens), keys, int(new[-1]))
    torch.cuda.synchronize()
    assert mla.mla_get_device_error() == 0
    flat, left = keys.view(-1, 576), torch.ones(n_pages * ps // 64, dtype=torch.bool, device="cuda")
    for s, l in enumerate(lens):
        lo, hi = (l - news[s]) // 64, l // 64
        if lo >= hi:
            continue
        x = rows[int(cu[s]) + 64 * lo:int(cu[s]) + 64 * hi].double().view(-1, 64, 576)
        j = torch.arange(lo, hi, device="cuda")
        slot = table[s, j * 64 // ps].long() * (ps // 64) + j % (ps // 64)
        tol = 64 * 2.0 ** -24 * x.abs().mean(1) + 2.0 ** -11 * x.mean(1).abs() + 2.0 ** -25     # as above
        assert ((flat[slot].double() - x.mean(1)).abs() <= tol).all()
        left[slot] = False
    assert (flat[left] == 7).all() and int(left.sum()) > 0


def test_block_keys_skips_bad_pages():
    b = Batch(9, False, 16, 64, [128], [128])
    keys = torch.full((b.n_pages, 1, 576), 7.0, dtype=torch.float16, device="cuda")
    for bad in (-1, b.n_pages):
        table = full_table(b)
        table[0, 0] = bad
        keys.fill_(7.0)
        mla.mla_paged_block_keys(b.pages_dev(), table, i32(b.cu), i32(b.lens), keys, b.T)
        torch.cuda.synchronize()
        assert mla.mla_get_device_error() == INVALID
        assert int((keys != 7).any(-1).sum()) == 1        # the other block's


# ---------------------------------------------------------------------------
# scores
# ---------------------------------------------------------------------------
@pytest.mark.parametrize("H", [16, 48, 112, 128])
@pytest.mark.parametrize("ps,news,lens,pad,width", [
    (64, [1], [1], 0, 1), (64, [1], [65], 0, 5), (128, [1, 0, 1, 1], [8300, 0, 63, 16385], 2, 257),
    (64, [70, 3, 1], [70, 400, 129], 1, 7), (256, [300], [8500], 0, 133), (4096, [9, 40], [20000, 16384 + 40], 0, 313),
    (64, [1] * 40, [64 * k + 1 for k in range(40)], 0, 45), (64, [0, 3, 0, 0], [0, 9000, 5, 0], 0, 150),
    (128, [700, 1, 333], [30000, 20000, 400], 1, 480)])
def test_block_scores(H, ps, news, lens, pad, width):
    b = Batch(10, False, H, ps, news, lens, pad=pad)
    rng = np.random.default_rng(11)
    keys = torch.full((b.n_pages, ps // 64, 576), float("nan"), dtype=torch.float16, device="cuda")   # not to be looked at
    per, kv = ps // 64, []
    table = b.table.copy()
    for s in range(b.B):
        m = max(0, (b.lens[s] - 1) // 64) if b.news[s] else 0
        k = (rng.standard_normal((m, 576)) * 0.3).astype(np.float16)
        for j in range(m):
            page = int(b.row_ids[s][64 * j]) // ps
            table[s, j // per] = page
            keys[page, j % per] = torch.from_numpy(k[j]).cuda()
        kv.append(k.astype(np.float64))
    wide = torch.full((b.T, width + 3), 7.0, device="cuda")
    scores = wide[:, :width]
    d = b.dev()
    mla.mla_paged_block_scores(d["q_lat"], d["q_pe"], keys, torch.from_numpy(table).cuda(), d["cu_q"], d["seq_len"], scores,
                               scale=SCALE)
    torch.cuda.synchronize()
    assert mla.mla_get_device_error() == 0
    assert (wide[:, width:] == 7).all() and (wide[b.cu[-1]:] == 7).all()
    got = host(scores)
    q = np.concatenate([b.q_lat, b.q_pe], -1).astype(np.float64)
    for s in range(b.B):
        lo, hi = b.cu[s], b.cu[s + 1]
        want, mag = BO.block_scores(q[lo:hi], kv[s], b.lens[s] - b.news[s], width, SCALE)
        hidden = np.isneginf(want)
        assert np.array_equal(np.isneginf(got[lo:hi]), hidden)
        # exact products; 36 accumulations of 16, cut off: 2^-23 of the largest partial sum and as much again within
        # each; the product with the scale
        tol = 2 * 36 * 2.0 ** -23 * mag + 2.0 ** -23 * np.abs(want)
        assert (np.abs(got[lo:hi][~hidden] - want[~hidden]) <= tol[~hidden]).all()


def test_block_scores_reports_short_rows_and_bad_pages():
    H, ps, L = 16, 64, 1000
    b = Batch(12, False, H, ps, [2], [L])
    keys = torch.ones(b.n_pages, 1, 576, dtype=torch.float16, device="cuda")
    d, table = b.dev(), full_table(b)
    whole = torch.empty(2, 15, device="cuda")
    mla.mla_paged_block_scores(d["q_lat"], d["q_pe"], keys, table, d["cu_q"], d["seq_len"], whole, scale=SCALE)
    torch.cuda.synchronize()
    assert mla.mla_get_device_error() == 0                # positions 998, 999: own block 15
    short = torch.empty(2, 14, device="cuda")
    mla.mla_paged_block_scores(d["q_lat"], d["q_pe"], keys, table, d["cu_q"], d["seq_len"], short, scale=SCALE)
    torch.cuda.synchronize()
    assert mla.mla_get_device_error() == INVALID
    assert torch.equal(short, whole[:, :14])
    table[0, 3] = b.n_pages + 5
    mla.mla_paged_block_scores(d["q_lat"], d["q_pe"], keys, table, d["cu_q"], d["seq_len"], short, scale=SCALE)
    torch.cuda.synchronize()
    assert mla.mla_get_device_error() == INVALID
    d["q_pe"][1, 5, 3] = 1e30
    mla.mla_paged_block_scores(d["q_lat"], d["q_pe"], keys, full_table(b), d["cu_q"], d["seq_len"], whole, scale=SCALE)
    torch.cuda.synchronize()
    assert mla.mla_get_device_error() == RANGE


# ---------------------------------------------------------------------------
# the choice
# ---------------------------------------------------------------------------
def choose(scores, news, lens, K, n_sink, n_local, T=None):
    cu = np.concatenate([[0], np.cumsum(news)])
    T = int(cu[-1]) if T is None else T
    blocks = torch.full((T, K), -7, dtype=torch.int32, device="cuda")
    counts = torch.full((T,), -7, dtype=torch.int32, device="cuda")
    mla.mla_paged_select_blocks(scores, i32(cu), i32(lens), blocks, counts, n_sink=n_sink, n_local=n_local)
    torch.cuda.synchronize()
    return blocks.cpu().numpy(), counts.cpu().numpy(), cu


@pytest.mark.parametrize("kind", ["random", "ties", "special"])
@pytest.mark.parametrize("K,n_sink,n_local", [(1, 0, 1), (2, 1, 1), (7, 2, 3), (64, 1, 2), (300, 0, 1)])
@pytest.mark.parametrize("news,lens,pad", [([1], [1], 0), ([1, 0, 70, 1], [64 * 31, 0, 300, 64 * 256 + 1], 2),
                                           ([3, 5], [64 * 300, 64 * 512 + 2], 0), ([2], [64 * 5000 + 1], 0)])
def test_select_blocks(kind, K, n_sink, n_local, news, lens, pad):
    rng = np.random.default_rng(13)
    T, W = sum(news) + pad, max(1, -(-max(lens) // 64)) + 3
    x = rng.standard_normal((T, W)).astype(np.float32)
    if kind == "ties":
        x = np.round(x).astype(np.float32) * np.where(rng.random((T, W)) < 0.5, 1, -0.0).astype(np.float32)
    elif kind == "special":
        x[rng.random((T, W)) < 0.3] = -np.inf
        x[rng.random((T, W)) < 0.05] = np.inf
        x[rng.random((T, W)) < 0.3] = np.nan
        x[rng.random((T, W)) < 0.1] = np.finfo(np.float32).min
    pos = np.concatenate([np.arange(l - n, l) for n, l in zip(news, lens)])
    wide = torch.from_numpy(np.concatenate([x, np.full((T, 5), 9, np.float32)], 1)).cuda()
    blocks, counts, cu = choose(wide[:, :W], news, lens, K, n_sink, n_local, T)
    assert mla.mla_get_device_error() == 0
    for t, p in enumerate(pos):
        want = BO.select(x[t], int(p), K, n_sink, n_local)
        assert counts[t] == len(want)
        assert np.array_equal(blocks[t, :len(want)], want) and (blocks[t, len(want):] == -1).all(), t
    assert (blocks[cu[-1]:] == -7).all() and (counts[cu[-1]:] == -7).all()


def test_select_blocks_reports_tokens_without_scores():
    scores = torch.randn(2, 10, device="cuda")
    blocks, counts, _ = choose(scores, [2], [641], 4, 1, 1)
    assert mla.mla_get_device_error() == INVALID
    assert list(blocks[1]) == [-1] * 4 and counts[1] == 0
    assert counts[0] == 4 and blocks[0, 0] == 0 and blocks[0, 3] == 9


def scores_of_kind(rng, kind, W, own, best):
    """A row of W scores for a token whose own block is ``own``; in runs, ``best`` neighbours before it stand out."""
    x = rng.standard_normal(W).astype(np.float32)
    if kind == "ties":
        x = np.round(2 * x)
    elif kind == "special":
        x[rng.random(W) < 0.3] = -np.inf
        x[rng.random(W) < 0.02] = np.inf
        x[rng.random(W) < 0.3] = np.nan
    elif kind == "rising":                               # of either sign
        x = np.linspace(-1, 1, W, dtype=np.float32)
    elif kind == "falling":
        x = np.linspace(-1, -5, W, dtype=np.float32)
    elif kind in ("run", "passage"):                     # neighbours around 0 or -2 above the rest
        n = min(best, own)
        at = int(rng.integers(0, own - n + 1))
        x = x - 20
        x[at:at + n] = (0 if kind == "run" else -2) + rng.standard_normal(n)
    elif kind == "same":
        x[:] = -0.0 if rng.random() < 0.5 else 3.0
    return x


@pytest.mark.parametrize("R", [1, 29, 31, 32, 33, 61, 63, 64, 65, 300])
@pytest.mark.parametrize("longest", [700, 1024, 1025, 2048])
def test_select_blocks_of_many_tokens(R, longest):
    """More tokens than a block of threads each is taken for: rows of each kind, long ones and such that have a few more
    candidates than are taken; nothing else is written."""
    kinds = ["random", "ties", "special", "rising", "falling", "run", "passage", "same"]
    n_sink, n_local = 1, 2
    K, many = R + n_sink + n_local, 8 * torch.cuda.get_device_properties(0).multi_processor_count
    # own blocks up to the row's last, around R candidates, and the first ones
    news, lens = [many // 2, 0, many // 2, 64 * 4 + 9, 70], [64 * longest, 0, 64 * (longest * 3 // 4) + 5, 64 * (R + 5) + 1, 70]
    lens = [min(n, 64 * longest) for n in lens]
    cu, pad = np.concatenate([[0], np.cumsum(news)]), 3
    T, W, rng = sum(news) + pad, longest, np.random.default_rng(41)
    assert T > many
    pos = np.concatenate([np.arange(l - n, l) for n, l in zip(news, lens)])
    x = np.full((T, W + 5), 1e30, np.float32)
    for t, p in enumerate(pos):
        x[t, :W] = scores_of_kind(rng, kinds[t % len(kinds)], W, int(p) // 64, (32, 64, R)[t // len(kinds) % 3])
    around = 4096
    flat = torch.full((T * K + 2 * around,), -7, dtype=torch.int32, device="cuda")
    cflat = torch.full((T + 2 * around,), -7, dtype=torch.int32, device="cuda")
    blocks, counts = flat[around:-around].view(T, K), cflat[around:-around]
    mla.mla_paged_select_blocks(torch.from_numpy(x).cuda()[:, :W], i32(cu), i32(lens), blocks, counts, n_sink=n_sink,
                                n_local=n_local)
    torch.cuda.synchronize()
    assert mla.mla_get_device_error() == 0
    for f in (flat, cflat):
        assert (f[:around] == -7).all() and (f[-around:] == -7).all()
    blocks, counts = blocks.cpu().numpy(), counts.cpu().numpy()
    assert (blocks[len(pos):] == -7).all() and (counts[len(pos):] == -7).all()
    for t, p in enumerate(pos):
        own = int(p) // 64
        forced = [j for j in range(own + 1) if j < n_sink or j > own - n_local]
        rest = np.arange(n_sink, max(n_sink, own - n_local + 1))
        rest = rest[np.argsort(-x[t, rest], kind="stable")]          # (NaN comes last)
        want = np.sort(np.concatenate([forced, rest[:K - len(forced)]])).astype(np.int32)
        if t % 97 == 0:
            assert np.array_equal(want, BO.select(x[t, :W], int(p), K, n_sink, n_local))
        assert counts[t] == len(want), t
        assert np.array_equal(blocks[t, :len(want)], want) and (blocks[t, len(want):] == -1).all(), (t, kinds[t % len(kinds)])


# ---------------------------------------------------------------------------
# attention over listed blocks
# ---------------------------------------------------------------------------
class Listed(Batch):
    """A batch whose tokens list blocks: a mode's, or what ``lists`` (one a token) says.  Rows that no token sees hold
    NaN, and pages without any have no table entry."""

    def __init__(self, seed, e4m3, H, ps, news, lens, K, mode="random", pad=0, lists=None, **kw):
        super().__init__(seed, e4m3, H, ps, news, lens, pad=pad, **kw)
        rng = np.random.default_rng(seed + 100)
        self.blocks, self.counts = np.full((self.T, K), 99999999, np.int32), np.zeros(self.T, np.int32)
        bad = np.where(rng.random(self.table.shape) < 0.5, -1, 1 << 30).astype(np.int32)
        t = 0
        for b in range(self.B):
            seen = np.zeros(lens[b], bool)
            for i in range(news[b]):
                p = lens[b] - news[b] + i
                own = p // 64
                if lists is not None:
                    want = lists[t]
                elif mode == "random":                  # in any order, any number of them
                    want = rng.permutation(own + 1)[:rng.integers(0, K + 1)]
                else:                                   # all that there are, up to K, the own among them
                    want = np.sort(np.append(rng.permutation(own)[:K - 1], own))
                self.blocks[t, :len(want)], self.counts[t] = want, len(want)
                for j in want:
                    if 0 <= j <= own:
                        seen[64 * j:min(64 * j + 64, p + 1)] = True
                t += 1
            self.raw[self.row_ids[b][~seen]] = 0xFF
            used = np.unique(np.flatnonzero(seen) // ps)
            entries = bad[b].copy()
            entries[used] = self.table[b, used]
            self.table[b] = entries
        self.table = np.ascontiguousarray(self.table)

    def dev(self):
        return dict(super().dev(), blocks=torch.from_numpy(self.blocks).cuda(), counts=torch.from_numpy(self.counts).cuda())

    def ref(self):
        """(o, bound): as Batch.ref derives it, for the listed keys."""
        q = np.concatenate([self.q_lat.astype(np.float64), self.q_pe.astype(np.float64)], -1)
        o, tol = [], []
        for b in range(self.B):
            for i in range(self.news[b]):
                t, p = self.cu[b] + i, self.lens[b] - self.news[b] + i
                lst = [j for j in self.blocks[t, :self.counts[t]] if 0 <= j <= p // 64]
                x, a, n = BO.attend_blocks(q[t], self.rows[b], p, lst, SCALE)
                o.append(x)
                tol.append((2.0 ** -11 + 2.0 ** -12) * a + 2.0 ** -11 * np.abs(x) + 2.0 ** -24
                           + 2.0 ** -25 * n * np.abs(self.rows[b]).max())
        return np.array(o), np.array(tol)


def attend(b, d=None, out=None, **kw):
    d = d or b.dev()
    out = torch.full((b.T, b.H, 512), float("nan"), dtype=torch.float16, device="cuda") if out is None else out
    mla.mla_attn_paged_blocks(d["q_lat"], d["q_pe"], d["pages"], d["block_table"], d["cu_q"], d["seq_len"], d["blocks"],
                              d["counts"], out, scale=SCALE, **kw)
    return out


def check(b, out, status=0):
    torch.cuda.synchronize()
    assert mla.mla_get_device_error() == status
    got = host(out)
    ref, tol = b.ref()
    n = b.cu[-1]
    assert np.isfinite(got[:n]).all()
    off = np.abs(got[:n] - ref) / tol
    assert off.max() <= 1.0, f"{off.max():.2f} of the bound at {np.unravel_index(off.argmax(), off.shape)}"
    assert np.isnan(got[n:]).all()


@pytest.mark.parametrize("e4m3", [False, True])
@pytest.mark.parametrize("H,ps,news,lens,K,mode,pad", [
    (16, 64, [1], [1], 1, "all", 0), (16, 64, [1], [65], 4, "all", 0), (128, 64, [1], [5000], 40, "all", 0),
    (128, 128, [1, 0, 1, 1], [700, 0, 64, 2049], 5, "random", 2), (64, 64, [1] * 9, [300 + 67 * k for k in range(9)], 3, "all", 0),
    (32, 256, [70, 3, 1], [70, 400, 129], 4, "random", 1), (128, 64, [33], [3000], 17, "all", 0),
    (48, 4096, [9, 40], [5000, 4136], 33, "random", 0), (32, 64, [0, 3, 0, 0], [0, 900, 5, 0], 4, "random", 0), (112, 64, [130], [131], 3, "all", 3), (16, 64, [260], [700], 2, "random", 0)])
def test_attention_over_listed_blocks(e4m3, H, ps, news, lens, K, mode, pad):
    b = Listed(14, e4m3, H, ps, news, lens, K, mode, pad)
    check(b, attend(b))


@pytest.mark.parametrize("e4m3", [False, True])
def test_tokens_without_blocks_get_zeros(e4m3):
    b = Listed(15, e4m3, 128, 64, [3, 1, 1], [200, 500, 64], 4, lists=[[], [2, 0], [], [], [0]])
    out = attend(b)
    check(b, out)
    assert (out[[0, 2, 3]] == 0).all()


def test_many_tokens_without_blocks():
    """Pieces of nothing beside pieces of much: a cluster's share starts and ends in either."""
    lists = [[] if t % 3 else list(range(t % 50)) for t in range(200)]
    b = Listed(16, False, 16, 64, [200], [3400], 50, lists=lists)
    check(b, attend(b))


@pytest.mark.parametrize("e4m3", [False, True])
def test_a_block_listed_twice_counts_twice(e4m3):
    b = Listed(17, e4m3, 64, 64, [2], [400], 8, lists=[[1, 1, 6, 0], [6, 6, 6, 2, 2]])
    check(b, attend(b))


@pytest.mark.parametrize("e4m3", [False, True])
def test_bad_entries_add_nothing_and_are_reported(e4m3):
    lists = [[0, -1, 3], [700, 2], [-5], [1 << 30, 4, -(1 << 31), 0]]
    for news, lens in (([4], [320]), ([1, 1, 1, 1], [300, 320, 100, 319])):
        b = Listed(18, e4m3, 128, 64, news, lens, 6, lists=lists)
        check(b, attend(b), INVALID)
    # only bad ones, many of them, in blocks that cluster boundaries cut
    b = Listed(19, e4m3, 128, 64, [1, 1], [300, 300], 400, lists=[[-1] * 400, [0, 1]])
    out = attend(b)
    check(b, out, INVALID)
    assert (out[0] == 0).all()


def test_counts_outside_the_list_are_reported():
    b = Listed(20, False, 16, 64, [2], [400], 3, lists=[[0, 1, 2], [3]])
    d = b.dev()
    d["counts"] += torch.tensor([5, -9], dtype=torch.int32, device="cuda")
    out = attend(b, d)
    b.counts[:] = [3, 0]
    check(b, out, INVALID)


def test_bad_pages_are_reported():
    b = Listed(21, False, 16, 64, [1, 1], [400, 300], 3, lists=[[0, 5], [1, 4]])
    d = b.dev()
    good = attend(b, d).clone()
    d["block_table"][0, 5] = b.n_pages
    out = attend(b, d)
    torch.cuda.synchronize()
    assert mla.mla_get_device_error() == INVALID
    assert torch.equal(out[1], good[1])                    # the other sequence is as usual


@pytest.mark.parametrize("e4m3", [False, True])
@pytest.mark.parametrize("K,lens", [(1024, [65536]), (700, [44800, 40000])])
def test_long_lists(e4m3, K, lens):
    """Every block of a context, the longest list among them: the whole attention."""
    b = Listed(22, e4m3, 16, 64, [1] * len(lens), lens, K, lists=[list(range(l // 64)) for l in lens])
    out = attend(b)
    check(b, out)
    d = b.dev()
    dense = torch.empty_like(out)
    mla.mla_attn_paged(d["q_lat"], d["q_pe"], d["pages"], d["block_table"], d["cu_q"], d["seq_len"], dense, scale=SCALE)
    torch.cuda.synchronize()
    assert mla.mla_get_device_error() == 0
    ref, tol = b.ref()
    assert (np.abs(host(out) - host(dense)) <= 2 * tol).all()


@pytest.mark.parametrize("e4m3", [False, True])
@pytest.mark.parametrize("H", [16, 48, 64])
def test_neighbours_with_lists_of_their_own(e4m3, H):
    """Chunks in which tokens share blocks of 128 rows: lists that agree, differ, are empty, name a block again or no
    block, and tiles whose later rows only tokens see that do not list them."""
    lists = [[0], [1, 0], [], [0, 1], [1, 1, 0, 1], [0], [], [1], [0, 0], [1], [1, 0], [0]]
    for K in (5, 400):
        b = Listed(31, e4m3, H, 64, [12], [70], K, lists=lists)       # positions 58 .. 69: up to 63, block 1 is ahead
        check(b, attend(b), INVALID)
    lists = [list(range(t % 5)) + [7 + t % 3] for t in range(60)]
    for K in (9, 64):                    # (long rows of short lists: enough entries to go in groups)
        b = Listed(32, e4m3, H, 128, [37, 2, 21], [700, 650, 900], K, lists=lists, pad=1)
        check(b, attend(b))
    lists[10], lists[41] = [-1, 3, 1 << 25], [3, 50, 3, 3, 2]
    for K in (9, 64):
        b = Listed(33, e4m3, H, 128, [37, 2, 21], [700, 650, 900], K, lists=lists, pad=1)
        check(b, attend(b), INVALID)


@pytest.mark.parametrize("H", [16, 64, 128])
@pytest.mark.parametrize("lens", [[600, 5000, 25000], [600, 640, 700], [30000, 26000, 25000]], ids=["some", "all", "none"])
def test_e4m3_chunks_converted_beforehand_or_not(H, lens):
    """Enough entries that sequences whose rows are read often are converted before the attention: some of them, all,
    none."""
    news = [80, 3 if lens[1] > 700 else 70, 40]
    pos = [l - n + i for n, l in zip(news, lens) for i in range(n)]
    lists = [sorted({(5 * t) % (p // 64 + 1), p // 64, 0, (t // 3) % (p // 64 + 1)}) for t, p in enumerate(pos)]
    b = Listed(37, True, H, 128, news, lens, 64, lists=lists, pad=1)
    check(b, attend(b))


@pytest.mark.parametrize("H,K,news,lens", [
    (16, 256, [300, 300], [60000, 69500]),       # both converted, with a few tiles' room behind them for the lists
    (16, 256, [300, 300], [60000, 71000]),       # the second one's rows and the lists do not fit
    (64, 1024, [900, 120], [100000, 22700]), (64, 1024, [900, 120], [100000, 31000])], ids=str)
def test_converted_rows_and_lists_share_the_workspace(H, K, news, lens):
    """Pages that stand in for many of a context's; the room for converted rows full to the lists that lie behind them."""
    rng, ps = np.random.default_rng(44), 4096
    lat, rope = bf16(rng.standard_normal((2 * ps, 512))), bf16(rng.standard_normal((2 * ps, 64)))
    raw = PO.pack_rows(lat, rope, True)
    rows, T = PO.row_values(raw, True), sum(news)
    table = rng.integers(0, 2, (2, -(-max(lens) // ps))).astype(np.int32)
    cu = np.concatenate([[0], np.cumsum(news)])
    g = torch.Generator(device="cuda").manual_seed(44)
    q_lat = torch.randn(T, H, 512, generator=g, device="cuda").half()
    q_pe = torch.randn(T, H, 64, generator=g, device="cuda").bfloat16()
    blocks, counts = np.full((T, K), -1, np.int32), rng.integers(0, 6, T).astype(np.int32)
    pos = np.concatenate([np.arange(l - n, l) for n, l in zip(news, lens)])
    for t, p in enumerate(pos):
        own = int(p) // 64
        near = np.clip([own, own - 1 - t % 3, t % 7, own // 2, own // 3 + t % 2], 0, own)
        blocks[t, :counts[t]] = near[:counts[t]]
    out = torch.full((T, H, 512), float("nan"), dtype=torch.float16, device="cuda")
    ws = torch.randint(0, 256, (mla.mla_paged_workspace_size(H) + 4096,), dtype=torch.uint8, device="cuda")
    behind = ws[-4096:].clone()
    mla.mla_attn_paged_blocks(q_lat, q_pe, torch.from_numpy(raw).cuda().view(2, ps, -1), i32(table), i32(cu), i32(lens),
                              i32(blocks), i32(counts), out, workspace=ws[:-4096], scale=SCALE)
    torch.cuda.synchronize()
    assert mla.mla_get_device_error() == 0 and torch.equal(ws[-4096:], behind)
    assert out.isfinite().all()
    for t in range(0, T, 13):
        lst, s, p = blocks[t, :counts[t]], int(t >= cu[1]), int(pos[t])
        q = np.concatenate([host(q_lat[t]), host(q_pe[t])], -1)
        if not len(lst):
            assert (out[t] == 0).all()
            continue
        keys = np.concatenate([np.arange(64 * j, min(64 * j + 64, p + 1)) for j in lst])
        r = rows[table[s, keys // ps] * ps + keys % ps]
        x = SCALE * (q @ r.T)
        w = np.exp(x - x.max(-1, keepdims=True))
        w /= w.sum(-1, keepdims=True)
        want, a = w @ r[:, :512], w @ np.abs(r[:, :512])
        tol = (2.0 ** -11 + 2.0 ** -12) * a + 2.0 ** -11 * np.abs(want) + 2.0 ** -24 + 2.0 ** -25 * len(keys) * np.abs(r).max()
        assert (np.abs(host(out[t]) - want) <= tol).all(), t


@pytest.mark.parametrize("e4m3", [False, True])
@pytest.mark.parametrize("H,n", [(16, 40), (64, 40), (128, 3), (16, 600)])
def test_decreasing_offsets_are_reported(e4m3, H, n):
    """Outputs are undefined then; the calls end, inside their memory, and the next ones are as ever."""
    lists = [[t % 5, 7] for t in range(3 * n)]
    b = Listed(38, e4m3, H, 64, [n, n, n], [1400, 1200, 1300], 96, lists=lists)
    d = b.dev()
    ws = torch.randint(0, 256, (mla.mla_paged_workspace_size(H),), dtype=torch.uint8, device="cuda")
    scores, keys = torch.empty(b.T, 23, device="cuda"), torch.zeros(b.n_pages, 1, 576, dtype=torch.float16, device="cuda")
    blocks, counts = torch.empty(b.T, 4, dtype=torch.int32, device="cuda"), torch.empty(b.T, dtype=torch.int32, device="cuda")
    full = full_table(b)
    for cu in ([0, 2 * n, n, 3 * n], [3 * n, 2 * n, n, 0], [0, -5, n, 2 * n], [n, 0, 3 * n, 3 * n], [0, n, 1 << 30, 3 * n]):
        bad = dict(d, cu_q=i32(cu))
        attend(b, bad, workspace=ws)
        mla.mla_paged_block_scores(d["q_lat"], d["q_pe"], keys, full, i32(cu), d["seq_len"], scores, scale=SCALE)
        mla.mla_paged_select_blocks(scores, i32(cu), d["seq_len"], blocks, counts, n_sink=1, n_local=1)
        mla.mla_paged_block_keys(d["pages"], full, i32(cu), d["seq_len"], keys, b.T)
        torch.cuda.synchronize()
        assert mla.mla_get_device_error() == INVALID
    check(b, attend(b, d, workspace=ws))


@pytest.mark.parametrize("e4m3", [False, True])
@pytest.mark.parametrize("word", [1, 63, 161, 299])
def test_decreasing_offsets_read_no_lists_of_their_own(e4m3, word):
    """A workspace in which every entry that is not written names a key within a block, and sequences of two tokens whose
    pages are all of the pool."""
    n, L, K, H = 60, 300, 64, 16
    lists = [[t % 5, 4] for t in range(2 * n)]
    b = Listed(47, e4m3, H, 64, [2] * n, [L] * n, K, lists=lists)
    d = b.dev()
    full, raw = full_table(b), torch.zeros_like(d["pages"].view(torch.uint8))
    ws = torch.full((mla.mla_paged_workspace_size(H) // 4,), word, dtype=torch.int32, device="cuda").view(torch.uint8)
    up, down = list(range(0, 2 * n + 1, 2)), list(range(2 * n, -1, -2))
    for cu in (down, up[:31][::-1] + up[31:], [x ^ 2 for x in up[:-1]] + up[-1:], [x ^ 1 for x in up]):
        attend(b, dict(d, cu_q=i32(cu), block_table=full, pages=raw.view(d["pages"].dtype).view(d["pages"].shape)), workspace=ws)
        torch.cuda.synchronize()
        assert mla.mla_get_device_error() == INVALID
    check(b, attend(b, d, workspace=ws))


def test_counts_outside_the_lists_of_a_group_are_reported():
    lists = [[t % 6] for t in range(600)]
    lists[:5] = [[0, 1, 2], [3], [1], [], [0, 4]]
    b = Listed(34, False, 16, 64, [600], [1000], 3, lists=lists)
    d = b.dev()
    d["counts"][:2] += torch.tensor([5, -9], dtype=torch.int32, device="cuda")
    out = attend(b, d)
    b.counts[1] = 0
    check(b, out, INVALID)


def test_more_lists_than_the_workspace_groups():
    lists = [[(7 * t) % 30, 30 + t % 3][:1 + t % 2] for t in range(2100)]
    b = Listed(35, False, 16, 64, [2100], [4100], 1024, lists=lists)
    check(b, attend(b), INVALID)         # (block 32 is ahead of the first 48 tokens)


@pytest.mark.parametrize("H,K", [(16, 4), (16, 1024), (128, 4)])
def test_contexts_past_a_million_rows(H, K):
    """Two pages stand in for all of a context's; lists of few entries, in rows that are short and long."""
    rng, L, n = np.random.default_rng(36), 1_100_003, 3
    rows = rng.standard_normal((8192, 576)).astype(np.float16)
    table = rng.integers(0, 2, (1, -(-L // 4096))).astype(np.int32)
    lists = [[17000, 5, 16383, 17187], [16384, 5, 0], [17187, 16385, 5, 40]]
    q_lat = rng.standard_normal((n, H, 512)).astype(np.float16)
    q_pe = bf16(rng.standard_normal((n, H, 64)))
    blocks = np.full((n, K), -1, np.int32)
    for t, x in enumerate(lists):
        blocks[t, :len(x)] = x
    out = torch.empty(n, H, 512, dtype=torch.float16, device="cuda")
    mla.mla_attn_paged_blocks(torch.from_numpy(q_lat).cuda(), torch.from_numpy(q_pe).bfloat16().cuda(),
                              torch.from_numpy(rows).cuda().view(2, 4096, 576), i32(table), i32([0, n]), i32([L]),
                              i32(blocks), i32([len(x) for x in lists]), out, scale=SCALE)
    torch.cuda.synchronize()
    assert mla.mla_get_device_error() == 0
    q = np.concatenate([q_lat, q_pe], -1).astype(np.float64)
    for t, lst in enumerate(lists):
        p = L - n + t
        keys = np.concatenate([np.arange(64 * j, min(64 * j + 64, p + 1)) for j in lst])
        r = rows[table[0, keys // 4096] * 4096 + keys % 4096].astype(np.float64)
        s = SCALE * (q[t] @ r.T)
        w = np.exp(s - s.max(-1, keepdims=True))
        w /= w.sum(-1, keepdims=True)
        want, a = w @ r[:, :512], w @ np.abs(r[:, :512])
        tol = (2.0 ** -11 + 2.0 ** -12) * a + 2.0 ** -11 * np.abs(want) + 2.0 ** -24 + 2.0 ** -25 * len(keys) * np.abs(r).max()
        assert (np.abs(host(out[t]) - want) <= tol).all()


def test_rows_at_far_addresses():
    """A pool past 4 GB: pages at its end."""
    b = Listed(23, False, 16, 256, [1, 2], [900, 700], 3, "all")
    far = 4 << 30
    n = far // (256 * 1152) + b.n_pages + 1
    pages = torch.empty(n, 256, 576, dtype=torch.float16, device="cuda")
    d = b.dev()
    pages[n - b.n_pages:] = d["pages"]
    d["block_table"] = torch.where((d["block_table"] >= 0) & (d["block_table"] < b.n_pages), d["block_table"] + (n - b.n_pages),
                                   d["block_table"])
    d["pages"] = pages
    check(b, attend(b, d))
    # their mean rows, too
    keys = torch.zeros(n, 4, 576, dtype=torch.float16, device="cuda")
    full = i32(np.array([[n - b.n_pages + int(b.row_ids[s][p]) // 256 if p < b.lens[s] else -1
                          for p in range(0, 1024, 256)] for s in range(2)]))
    mla.mla_paged_block_keys(pages.nan_to_num_(0.0), full, i32([0, 900, 1600]), i32(b.lens), keys, 1600)
    torch.cuda.synchronize()
    assert mla.mla_get_device_error() == 0
    assert int((keys != 0).any(-1).sum()) <= 14 + 10 and (keys[:n - b.n_pages] == 0).all()


def test_the_same_call_gives_the_same_bits():
    b = Listed(24, True, 128, 64, [40, 1, 3], [2000, 900, 4000], 12, "all")
    d = b.dev()
    out = attend(b, d)
    ws = torch.randint(0, 256, (mla.mla_paged_workspace_size(128),), dtype=torch.uint8, device="cuda")
    for _ in range(3):
        again = attend(b, d, workspace=ws)
        torch.cuda.synchronize()
        assert torch.equal(out.view(torch.int16), again.view(torch.int16))
    assert mla.mla_get_device_error() == 0


# ---------------------------------------------------------------------------
# together
# ---------------------------------------------------------------------------
class Step:
    """A model's weights and a paged cache that sequences grow in."""

    def __init__(self, seed, H, ps, B, longest, e4m3, T):
        self.rng = np.random.default_rng(seed)
        self.H, self.ps, self.e4m3, self.B = H, ps, e4m3, B
        g = lambda *s, k=1.0: torch.from_numpy((self.rng.standard_normal(s) * k).astype(np.float32)).bfloat16().cuda()  # noqa: E731
        self.g = g
        self.wk, self.wv = g(H, 128, 512, k=128 ** -0.5), g(H, 512, 128, k=512 ** -0.5)
        self.qw, self.kw = 1 + g(192, k=0.1), 1 + g(512, k=0.1)
        width = -(-longest // ps)
        self.table = i32(self.rng.permutation(B * width + 1)[:B * width].reshape(B, width))
        self.pages = mla.paged_pages(B * width + 1, ps, e4m3)
        self.pages.view(torch.uint8).fill_(0xFF)
        self.keys = mla.paged_block_keys(self.pages).fill_(float("nan"))
        self.n_scores = width * ps // 64

    def inputs(self, T):
        both = self.g(T, self.H * 192 + 576)
        return both[:, :self.H * 192].unflatten(1, (self.H, 192)), both[:, self.H * 192:]

    def go(self, q, kv, cu, lens, K=4, n_sink=1, n_local=2, **kw):
        return mla.mla_paged_sparse_step(q, kv, self.qw, self.kw, self.wk, self.wv, self.pages, self.keys, self.table, cu,
                                         lens, n_blocks=K, n_sink=n_sink, n_local=n_local, eps=EPS, freq_base=FB,
                                         freq_scale=FS, scale=SCALE, **kw)


@pytest.mark.parametrize("e4m3", [False, True])
def test_steps_of_a_batch(e4m3):
    """Prompts in chunks, then single tokens: each call's output against the definition on the call before's."""
    H, ps, B = 32, 128, 3
    m = Step(25, H, ps, B, 1300, e4m3, 0)
    lens = np.zeros(B, int)
    for news, pad in (([700, 0, 130], 0), ([300, 64, 1], 3), ([1, 1, 1], 0), ([1, 63, 62], 1), ([1, 1, 1], 0)):
        lens = lens + news
        T = sum(news) + pad
        cu = np.concatenate([[0], np.cumsum(news)])
        q, kv = m.inputs(T)
        r = m.go(q, kv, i32(cu), i32(lens))
        torch.cuda.synchronize()
        assert mla.mla_get_device_error() == 0
        flat = m.pages.view(torch.uint8).reshape(-1, PO.ROW8 if e4m3 else 2 * PO.ROW).cpu().numpy()
        table = m.table.cpu().numpy()
        q_lat, q_pe, keys = host(r.q_lat), host(r.q_pe), host(m.keys).reshape(-1, 576)
        scores, blocks, counts, o_lat = host(r.scores), r.blocks.cpu().numpy(), r.counts.cpu().numpy(), host(r.o_lat)
        qx = np.concatenate([q_lat, q_pe], -1)
        n = cu[-1]
        x = BO.rms(host(q[:n]), host(m.qw), EPS)
        assert np.abs(host(r.q_nope[:n]) - x[..., :128]).max() <= 2.0 ** -7 * np.abs(x).max()
        for s in np.flatnonzero(lens):
            p = np.arange(lens[s])
            slot = table[s, p // ps].astype(np.int64) * ps + p % ps
            rows = PO.row_values(flat[slot], e4m3)
            assert np.isfinite(rows).all()
            means = BO.mean_rows(rows)
            k = keys[slot[:len(means) * 64:64] // 64]
            assert (np.abs(k - means) <= 2.0 ** -10 * np.abs(rows).max()).all()        # old blocks' among them
            want, mag = BO.block_scores(qx[cu[s]:cu[s + 1]], k, lens[s] - news[s], m.n_scores, SCALE)
            for i in range(news[s]):
                t, pos = cu[s] + i, lens[s] - news[s] + i
                fine = ~np.isneginf(want[i])
                assert np.array_equal(np.isneginf(scores[t]), ~fine)
                assert (np.abs(scores[t][fine] - want[i][fine]) <= 2.0 ** -16 * mag[i][fine]).all()
                lst = BO.select(scores[t], int(pos), 4, 1, 2)
                assert np.array_equal(blocks[t, :counts[t]], lst)
                if i % 37 and news[s] > 1:
                    continue
                o, a, c = BO.attend_blocks(qx[t], rows, int(pos), lst, SCALE)
                tol = 2.0 ** -10 * (a + np.abs(o)) + 2.0 ** -24 + 2.0 ** -25 * c * np.abs(rows).max()
                assert (np.abs(o_lat[t] - o) <= tol).all()
        o = O.late_decompress(o_lat[:n].astype(np.float64), host(m.wv))
        d = np.abs(host(r.o[:n]) - o)
        assert d.max() <= 1e-2 * np.abs(o).max() and d.mean() <= 2e-3 * np.abs(o).mean()


def test_steps_captured_and_replayed_on_streams():
    """A decode step captured on a side stream, twice with workspaces of their own, replayed side by side on new
    inputs, gives the eager call's bits."""
    from mla_latent_kv_lat_gb300 import pipeline as P
    H, ps, B, K = 16, 64, 4, 5
    sets = []
    for seed in (26, 27):
        m = Step(seed, H, ps, B, 900, False, B)
        lens = np.array([500, 64, 700, 63])
        q, kv = m.inputs(sum(lens))
        m.go(q, kv, i32(np.concatenate([[0], np.cumsum(lens)])), i32(lens), K)
        cu, ln = i32(np.arange(B + 1)), i32(lens)
        q, kv = m.inputs(B)
        bufs = P.sparse_buffers(B, H, m.n_scores, K)
        sets.append((m, q, kv, cu, ln, bufs, lens))
    torch.cuda.synchronize()
    graphs, streams = [], []
    for m, q, kv, cu, ln, bufs, lens in sets:
        s, g = torch.cuda.Stream(), torch.cuda.CUDAGraph()
        ln += 1
        s.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(s):
            m.go(q, kv, cu, ln, K, bufs=bufs)
        s.synchronize()
        with torch.cuda.graph(g, stream=s):
            m.go(q, kv, cu, ln, K, bufs=bufs)
        graphs.append(g)
        streams.append(s)
    want = []
    for m, q, kv, cu, ln, bufs, lens in sets:
        ln += 1                                          # the next token: lengths 502, 66, 702, 65
        a, b = m.inputs(B)
        q.copy_(a)
        kv.copy_(b)
        r = m.go(q, kv, cu, ln, K)
        want.append([x.clone() for x in (r.o, r.blocks, r.scores)])
    torch.cuda.synchronize()
    for _ in range(3):
        for g, s in zip(graphs, streams):
            with torch.cuda.stream(s):
                g.replay()
    torch.cuda.synchronize()
    assert mla.mla_get_device_error() == 0
    for (m, q, kv, cu, ln, bufs, lens), w in zip(sets, want):
        for x, y in zip((bufs.o, bufs.blocks, bufs.scores), w):
            assert torch.equal(x, y)


def test_a_step_on_a_stream_handle_of_its_own():
    H, B = 16, 2
    m = Step(28, H, 64, B, 300, True, B)
    lens = np.array([150, 200])
    q, kv = m.inputs(350)
    cu = i32([0, 150, 350])
    want = m.go(q, kv, cu, i32(lens))
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    for stream in (s, s.cuda_stream):
        got = m.go(q, kv, cu, i32(lens), stream=stream)
        s.synchronize()
        assert torch.equal(got.o, want.o) and torch.equal(got.blocks, want.blocks)
    assert mla.mla_get_device_error() == 0


def test_calls_agree_with_the_plain_append():
    """Weights of one, latents of mean square one: the normed append writes what mla_paged_append writes, to a rounding."""
    b = Batch(29, False, 16, 64, [70, 1], [200, 64])
    rng = np.random.default_rng(30)
    kv = torch.from_numpy(rng.choice([-1.0, 1.0], (b.T, 576)).astype(np.float32)).bfloat16().cuda()
    q = torch.zeros(b.T, 16, 192, dtype=torch.bfloat16, device="cuda")
    pages = [b.pages_dev().nan_to_num_(0.0) for _ in range(2)]
    one = torch.ones(512, dtype=torch.bfloat16, device="cuda")
    outs = [torch.empty(b.T, 16, n, dtype=torch.bfloat16, device="cuda") for n in (128, 64)]
    mla.mla_paged_norm_append(q, kv, None, one, pages[0], full_table(b), i32(b.cu), i32(b.lens), *outs, eps=1e-12)
    mla.mla_paged_append(kv[:, :512].contiguous(), kv[:, 512:].contiguous(), pages[1], full_table(b), i32(b.cu), i32(b.lens))
    torch.cuda.synchronize()
    assert mla.mla_get_device_error() == 0
    assert torch.equal(pages[0], pages[1])


def test_the_compiled_way_and_the_way_through_python_agree(monkeypatch):
    """Every paged call by the compiled module, which has to take it, and by the binding alone: the same bits."""
    from mla_latent_kv_lat_gb300 import binding as B
    H, T = 16, 90
    b = Listed(40, False, H, 64, [89, 1], [300, 500], 3, "all")
    d, full = b.dev(), full_table(b)
    rows = b.pages_dev().nan_to_num_(0.0)
    g = lambda *s, dt=torch.bfloat16: torch.randn(*s, device="cuda").to(dt)  # noqa: E731
    q, kv, qw, kw = g(T, H, 192), g(T, 576), g(192), g(512)
    c_kv, k_pe, keys = g(T, 512), g(T, 64), torch.zeros(b.n_pages, 1, 576, dtype=torch.float16, device="cuda")
    ws = torch.empty(mla.mla_paged_workspace_size(H), dtype=torch.uint8, device="cuda")
    cu, ln = d["cu_q"], d["seq_len"]

    def outs():
        e = lambda *s, dt=torch.float16: torch.zeros(*s, dtype=dt, device="cuda")  # noqa: E731
        return dict(pages=rows.clone(), q_nope=e(T, H, 128, dt=torch.bfloat16), q_pe=e(T, H, 64, dt=torch.bfloat16),
                    gathered=e(T, 576, dt=torch.bfloat16), keys=keys.clone(), scores=e(T, 8, dt=torch.float32),
                    blocks=e(T, 3, dt=torch.int32), counts=e(T, dt=torch.int32), o=e(T, H, 512), whole=e(T, H, 512))

    def calls(o, stream):
        ws_blocks = (d["blocks"], d["counts"])
        return [
            ("append", mla.mla_paged_append, (c_kv, k_pe, o["pages"], full, cu, ln, 1e4, 0.025, stream)),
            ("norm_append", mla.mla_paged_norm_append, (q, kv, qw, kw, o["pages"], full, cu, ln, o["q_nope"], o["q_pe"], 1e-6,
                                                        1e4, 0.025, stream)),
            ("gather", mla.mla_paged_gather, (o["pages"], full, ln - torch.diff(cu), cu, o["gathered"], stream)),
            ("block_keys", mla.mla_paged_block_keys, (o["pages"], full, i32([0, 300, 800]), ln, o["keys"], 800, stream)),
            ("block_scores", mla.mla_paged_block_scores, (d["q_lat"], d["q_pe"], o["keys"], full, cu, ln, o["scores"], SCALE,
                                                          stream)),
            ("select_blocks", mla.mla_paged_select_blocks, (o["scores"], cu, ln, o["blocks"], o["counts"], 1, 1, stream)),
            ("attn_blocks", mla.mla_attn_paged_blocks, (d["q_lat"], d["q_pe"], o["pages"], full, cu, ln, *ws_blocks, o["o"], ws, SCALE,
                                                        stream)),
            ("attn", mla.mla_attn_paged, (d["q_lat"], d["q_pe"], o["pages"], full, cu, ln, o["whole"], 0, 0, ws, SCALE, stream))]

    fast, slow, handle = outs(), outs(), outs()
    for name, _, args in calls(fast, None):
        assert getattr(B._fast(), name)(*args) == 0, name
    for _, fn, args in calls(handle, torch.cuda.current_stream().cuda_stream):
        fn(*args)
    monkeypatch.setattr(B, "_calls", B._Unbuilt())
    for _, fn, args in calls(slow, torch.cuda.current_stream()):
        fn(*args)
    torch.cuda.synchronize()
    assert mla.mla_get_device_error() == 0
    for k in fast:
        assert torch.equal(fast[k], slow[k]) and torch.equal(fast[k], handle[k]), k


def test_the_compiled_way_calls_the_library_without_the_interpreters_lock(tmp_path):
    """A stand-in for the library says whether its caller holds the lock (1) or not (0)."""
    import subprocess
    from mla_latent_kv_lat_gb300 import binding as B
    names = ("mla_paged_append", "mla_paged_gather", "mla_attn_paged", "mla_paged_norm_append", "mla_paged_block_keys",
             "mla_paged_block_scores", "mla_paged_select_blocks", "mla_attn_paged_blocks")
    src, lib = tmp_path / "stub.c", tmp_path / "stub.so"
    src.write_text("int PyGILState_Check(void);\n" + "".join(f"int {n}() {{ return PyGILState_Check(); }}\n" for n in names))
    subprocess.run(["gcc", "-shared", "-fPIC", "-o", str(lib), str(src)], check=True)
    H, T, bf, f16, i4 = 16, 2, torch.bfloat16, torch.float16, torch.int32
    z = lambda *s, dt=bf: torch.zeros(*s, dtype=dt, device="cuda")  # noqa: E731
    pages, table, cu, ln = z(3, 64, 576, dt=f16), z(1, 2, dt=i4), z(2, dt=i4), z(1, dt=i4)
    q_lat, q_pe, keys, scores = z(T, H, 512, dt=f16), z(T, H, 64), z(3, 1, 576, dt=f16), z(T, 5, dt=torch.float32)
    blocks, counts, ws = z(T, 3, dt=i4), z(T, dt=i4), z(64, dt=torch.uint8)
    fast = B._fast()
    fast.bind(str(lib))
    try:
        got = [fast.append(z(T, 512), q_pe[:, 0].contiguous(), pages, table, cu, ln, 1e4, 0.025, None),
               fast.gather(pages, table, None, cu, z(T, 576), None),
               fast.attn(q_lat, q_pe, pages, table, cu, ln, q_lat.clone(), 0, 0, ws, None, None),
               fast.norm_append(z(T, H, 192), z(T, 576), None, z(512), pages, table, cu, ln, z(T, H, 128), q_pe, 1e-6, 1e4, 0.025,
                                None),
               fast.block_keys(pages, table, cu, ln, keys, T, None),
               fast.block_scores(q_lat, q_pe, keys, table, cu, ln, scores, None, None),
               fast.select_blocks(scores, cu, ln, blocks, counts, 1, 1, None),
               fast.attn_blocks(q_lat, q_pe, pages, table, cu, ln, blocks, counts, q_lat.clone(), ws, None, None)]
    finally:
        fast.bind(B._build.LIB)
    assert got == [0] * len(names)


def test_the_compiled_way_and_the_way_through_python_refuse_alike(monkeypatch):
    """Every argument of every paged call replaced by what is not right: the same error by the same words, nothing written."""
    from mla_latent_kv_lat_gb300 import binding as B
    H, T, bf, f16, i4, f32, u8 = 16, 2, torch.bfloat16, torch.float16, torch.int32, torch.float32, torch.uint8
    z = lambda *s, dt=bf: torch.zeros(*s, dtype=dt, device="cuda")  # noqa: E731
    cache = dict(pages=z(3, 64, 576, dt=f16), block_table=z(1, 2, dt=i4))
    batch = dict(cu_q=z(2, dt=i4), seq_len=z(1, dt=i4))
    new = dict(cu_new=z(2, dt=i4), seq_len=z(1, dt=i4))
    q = dict(q_lat=z(T, H, 512, dt=f16), q_pe=z(T, H, 64))
    ws = z(mla.mla_paged_workspace_size(H), dt=u8)
    calls = [
        (mla.mla_paged_append, dict(c_kv=z(T, 512), k_pe=z(T, 64), **cache, **new, freq_base=1e4, freq_scale=0.025)),
        (mla.mla_paged_gather, dict(**cache, row0=z(1, dt=i4), cu_rows=z(2, dt=i4), out=z(T, 576))),
        (mla.mla_attn_paged, dict(**q, **cache, **batch, o_lat=z(T, H, 512, dt=f16), window=0, n_sink=0, workspace=ws)),
        (mla.mla_paged_norm_append, dict(q=z(T, H, 192), kv=z(T, 576), q_weight=z(192), kv_weight=z(512), **cache, **new,
                                         q_nope=z(T, H, 128), q_pe=z(T, H, 64), eps=1e-6, freq_base=1e4, freq_scale=0.025)),
        (mla.mla_paged_block_keys, dict(**cache, **new, block_keys=z(3, 1, 576, dt=f16), T=T)),
        (mla.mla_paged_block_scores, dict(**q, block_keys=z(3, 1, 576, dt=f16), block_table=cache["block_table"], **batch,
                                          scores=z(T, 5, dt=f32), scale=SCALE)),
        (mla.mla_paged_select_blocks, dict(scores=z(T, 5, dt=f32), **batch, blocks=z(T, 3, dt=i4), counts=z(T, dt=i4), n_sink=1,
                                           n_local=1)),
        (mla.mla_attn_paged_blocks, dict(**q, **cache, **batch, blocks=z(T, 3, dt=i4), counts=z(T, dt=i4),
                                         o_lat=z(T, H, 512, dt=f16), workspace=ws, scale=SCALE))]

    def wrong(name, t):
        if isinstance(t, torch.Tensor):
            other = f32 if t.dtype is not f32 else f16
            yield "type", t.to(other)
            yield "place", t.cpu()
            yield "none", 3.5
            if t is ws:
                yield "small", t[:4096]
                yield "odd", t[8:]
                return
            yield "more", torch.cat([t, t]) if t.dim() == 1 else torch.cat([t, t], -1)
            yield "flat", t.flatten() if t.dim() > 1 else t[None]
            if t.dim() > 1 and t.size(-1) > 1:
                yield "gaps", torch.cat([t, t], -1)[..., ::2]
            flat = torch.zeros(t.numel() + 1, dtype=t.dtype, device="cuda")
            if t.dtype in (bf, f16):
                yield "odd", flat[1:].view(t.shape)
        elif name in ("window", "n_sink", "n_local", "T"):
            yield "negative", -1
            yield "far", 1 << 31
        else:                                             # eps, frequencies, scale
            yield "zero", 0.0
            yield "negative", -1.0
            yield "nan", float("nan")
            yield "words", "1.5"

    def outcome(fn, kw):
        try:
            fn(**kw)
        except Exception as e:  # noqa: BLE001
            return type(e), str(e)
        return None

    fast, seen = B._fast(), 0
    assert not isinstance(fast, B._Unbuilt)
    for fn, kw in calls:
        assert outcome(fn, kw) is None, fn
        for name, t in kw.items():
            for what, bad in wrong(name, t):
                monkeypatch.setattr(B, "_calls", fast)
                got = outcome(fn, dict(kw, **{name: bad}))
                monkeypatch.setattr(B, "_calls", B._Unbuilt())
                want = outcome(fn, dict(kw, **{name: bad}))
                monkeypatch.setattr(B, "_calls", fast)
                assert got == want, (fn.__name__, name, what)
                seen += want is not None
    torch.cuda.synchronize()
    assert mla.mla_get_device_error() == 0 and seen > 200


@pytest.mark.parametrize("n_seqs", [400, 1500])
def test_batches_of_many_sequences(n_seqs):
    """More sequences than a block of threads has: every call against the definition, as above."""
    rng = np.random.default_rng(45)
    news = rng.choice([0, 1, 1, 1, 2, 5], n_seqs)
    lens = news + rng.integers(0, 150, n_seqs) * (rng.random(n_seqs) < 0.8)
    lens[::97] += 900
    news, lens = [int(x) for x in news], [int(x) for x in lens]
    test_block_scores(16, 64, news, lens, 3, 20)
    test_block_keys(False, 64, news, lens, 2)
    test_norm_append(True, 16, True, False, 64, news, lens, 1)
    for H, e4m3, K in ((16, False, 2), (128, True, 3)):
        b = Listed(46, e4m3, H, 64, news, lens, K, "random", 1)
        check(b, attend(b))
    K, W = 4, 20
    scores = rng.standard_normal((sum(news), W)).astype(np.float32)
    blocks, counts, cu = choose(torch.from_numpy(scores).cuda(), news, lens, K, 1, 1)
    assert mla.mla_get_device_error() == 0
    for t, p in enumerate(np.concatenate([np.arange(l - n, l) for n, l in zip(news, lens)])):
        want = BO.select(scores[t], int(p), K, 1, 1)
        assert counts[t] == len(want) and np.array_equal(blocks[t, :len(want)], want)
