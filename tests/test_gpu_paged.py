"""The paged latent cache on the GPU: rows written and read back bit for bit against the oracle, and attention over
pages (whole context, sliding window with sinks; one token a sequence, chunks, both mixed) against the 64-bit
definition, with a bound per value that follows from the arithmetic."""
import numpy as np
import pytest
import torch

import mla_latent_kv_lat_gb300 as mla
from mla_latent_kv_lat_gb300 import pipeline as P
from oracle import mla_oracle as O
from oracle import paged_oracle as PO
from tests.paged_util import SCALE, Batch, bf16

pytestmark = pytest.mark.gpu

INVALID, RANGE = -1, -7
FB, FS = float(np.float32(10000.0)), float(np.float32(0.025))


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


def run(b: Batch, d=None, out=None, **kw):
    d = d or b.dev()
    out = torch.full((b.T, b.H, 512), float("nan"), dtype=torch.float16, device="cuda") if out is None else out
    mla.mla_attn_paged(d["q_lat"], d["q_pe"], d["pages"], d["block_table"], d["cu_q"], d["seq_len"], out,
                       window=b.window, n_sink=b.n_sink, scale=SCALE, **kw)
    return out


def check(b: Batch, out):
    torch.cuda.synchronize()
    assert mla.mla_get_device_error() == 0
    got = out.float().cpu().numpy().astype(np.float64)
    ref, tol = b.ref()
    n = b.cu[-1]
    assert np.isfinite(got[:n]).all()
    off = np.abs(got[:n] - ref) / tol
    assert off.max() <= 1.0, f"{off.max():.2f} of the bound at {np.unravel_index(off.argmax(), off.shape)}"
    assert np.isnan(got[n:]).all()                      # rows behind the last sequence stay as they were


# ---------------------------------------------------------------------------
# writing and reading back
# ---------------------------------------------------------------------------
@pytest.mark.parametrize("e4m3", [False, True])
@pytest.mark.parametrize("ps,news,lens,pad", [
    (16, [1], [1], 0), (64, [1, 0, 3, 1], [700, 0, 3, 64], 2), (32, [130, 65, 1], [131, 1000, 33], 0),
    (256, [255, 300], [5000, 300], 5)])
def test_append_writes_rows_and_gather_reads_them(e4m3, ps, news, lens, pad):
    b = Batch(3, e4m3, 16, ps, news, lens, pad=pad)
    rng = np.random.default_rng(4)
    c_kv = bf16(rng.standard_normal((b.T, 512)) * np.exp(rng.uniform(-12, 9, (b.T, 1))))
    c_kv[0, :40] = 0.0                                   # a block of zeros and one that is half zero
    k_pe = bf16(rng.standard_normal((b.T, 64)))
    pages, table = b.pages_dev(), torch.from_numpy(b.table).cuda()
    for s in range(b.B):                                 # every page of the sequence in the table
        p = np.arange(0, b.lens[s], ps)
        table[s, :len(p)] = torch.from_numpy((b.row_ids[s][p] // ps).astype(np.int32)).cuda()
    mla.mla_paged_append(torch.from_numpy(c_kv).bfloat16().cuda(), torch.from_numpy(k_pe).bfloat16().cuda(), pages,
                         table, i32(b.cu), i32(b.lens), freq_base=FB, freq_scale=FS)
    torch.cuda.synchronize()
    assert mla.mla_get_device_error() == 0
    raw = pages.view(torch.uint8).reshape(b.raw.shape).cpu().numpy()
    want = b.raw.copy()
    for s in range(b.B):
        lo, hi = b.cu[s], b.cu[s + 1]
        pos = np.arange(b.lens[s] - b.news[s], b.lens[s])
        slot = b.row_ids[s][pos]
        rope = PO.rope_rows(k_pe[lo:hi], pos, FB, FS)
        want[slot] = PO.pack_rows(c_kv[lo:hi], rope, e4m3)
        o = 512 if e4m3 else 1024
        got_rope = np.ascontiguousarray(raw[slot, o:o + 128]).view(np.float16).astype(np.float64)
        # sine, cosine and the rotation in fp32 (a few 2^-24 of the pair's length), then one rounding to fp16
        pair = np.repeat(np.hypot(k_pe[lo:hi, 0::2], k_pe[lo:hi, 1::2]), 2, axis=1)
        assert (np.abs(got_rope - rope) <= 2.0 ** -11 * np.abs(rope) + 1e-6 * pair + 2.0 ** -25).all()
        want[slot, o:o + 128] = raw[slot, o:o + 128]
    assert np.array_equal(raw, want)                     # latents, codes, scales; no other byte touched
    # read back: the new rows and up to 70 before them
    back = [min(l, n + 70) for n, l in zip(b.news, b.lens)]
    row0 = [l - k for l, k in zip(b.lens, back)]
    cu_rows = np.concatenate([[0], np.cumsum(back)])
    slots = np.concatenate([b.row_ids[s][row0[s]:] for s in range(b.B)]).astype(int)
    vals = PO.row_values(want[slots], e4m3)
    for dt in (torch.float16, torch.bfloat16):
        out = torch.full((int(cu_rows[-1]) + 3, 576), 7.0, dtype=dt, device="cuda")
        mla.mla_paged_gather(pages, table, i32(row0), i32(cu_rows), out)
        torch.cuda.synchronize()
        assert mla.mla_get_device_error() == 0
        ref = torch.from_numpy(vals).to(torch.float32).to(dt)   # every row value is exact in fp32
        assert torch.equal(torch.nan_to_num(out[:-3].cpu(), 9.0), torch.nan_to_num(ref, 9.0))
        assert (out[-3:] == 7.0).all()


def test_append_at_far_positions_and_gather_from_zero():
    ps, L = 4096, 200001
    n_pages = -(-L // ps)
    pages = torch.zeros(n_pages, ps, 576, dtype=torch.float16, device="cuda")
    table = torch.arange(n_pages, dtype=torch.int32, device="cuda").flip(0)[None].contiguous()
    k_pe = bf16(np.random.default_rng(0).standard_normal((3, 64)))
    mla.mla_paged_append(torch.ones(3, 512, dtype=torch.bfloat16, device="cuda"),
                         torch.from_numpy(k_pe).bfloat16().cuda(), pages, table, i32([0, 3]), i32([L]))
    out = torch.empty(L, 576, dtype=torch.float16, device="cuda")
    mla.mla_paged_gather(pages, table, None, i32([0, L]), out)
    torch.cuda.synchronize()
    assert mla.mla_get_device_error() == 0
    assert (out[:-3] == 0).all() and (out[-3:, :512] == 1).all()
    ref = PO.rope_rows(k_pe, np.arange(L - 3, L), FB, FS)
    assert np.abs(out[-3:, 512:].cpu().numpy() - ref).max() <= 2.0 ** -11 * np.abs(ref).max() + 1e-5


@pytest.mark.parametrize("e4m3", [False, True])
def test_values_a_row_cannot_hold_are_reported(e4m3):
    pages = P.paged_pages(1, 16, e4m3)
    table = torch.zeros(1, 1, dtype=torch.int32, device="cuda")
    c = torch.ones(1, 512, dtype=torch.bfloat16, device="cuda")
    k = torch.ones(1, 64, dtype=torch.bfloat16, device="cuda")
    call = lambda: mla.mla_paged_append(c, k, pages, table, i32([0, 1]), i32([1]))   # noqa: E731
    call()
    assert mla.mla_get_device_error() == 0
    for bad in (1.0e5, float("inf"), float("nan")):
        c[0, 100] = bad
        call()
        assert mla.mla_get_device_error() == RANGE
        c[0, 100] = 57344.0                              # 448 * 2^7: the largest both types hold exactly
        call()
        assert mla.mla_get_device_error() == 0
        k[0, 5] = bad
        call()
        assert mla.mla_get_device_error() == RANGE
        k[0, 5] = 1.0


def test_bad_sequences_and_pages_are_skipped_and_reported():
    b = Batch(5, False, 16, 16, [2, 2, 2, 2], [40, 33, 20, 50])
    c_kv = torch.ones(8, 512, dtype=torch.bfloat16, device="cuda")
    k_pe = torch.ones(8, 64, dtype=torch.bfloat16, device="cuda")
    d = b.dev()
    for what in ("len", "neg", "page", "long"):
        lens, table = i32(b.lens), d["block_table"].clone()
        if what == "len":
            lens[1] = 1                                  # two new tokens, one row
        elif what == "neg":
            lens[1] = -5
        elif what == "long":
            lens[1] = b.width * 16 + 1
        else:
            table[1, 2] = b.n_pages                      # positions 32.. of sequence 1
        pages = d["pages"].clone()
        mla.mla_paged_append(c_kv, k_pe, pages, table, i32(b.cu), lens)
        assert mla.mla_get_device_error() == INVALID
        flat = pages.reshape(-1, 576)
        for s in (0, 2, 3):
            rows = torch.from_numpy(b.row_ids[s][b.lens[s] - 2:b.lens[s]]).cuda()
            assert (flat[rows, :512] == 1).all()
        # position 31 of sequence 1 is on the page before the bad one
        assert (flat[:, :512] == 1).all(1).sum() == (7 if what == "page" else 6)
        out = torch.full((b.T, 16, 512), 7.0, dtype=torch.float16, device="cuda")
        mla.mla_attn_paged(d["q_lat"], d["q_pe"], d["pages"], table, d["cu_q"], lens, out, scale=SCALE)
        assert mla.mla_get_device_error() == INVALID
        ref, tol = b.ref()
        got = out.float().cpu().numpy()
        for s in (0, 2, 3):
            lo, hi = b.cu[s], b.cu[s + 1]
            assert (np.abs(got[lo:hi] - ref[lo:hi]) <= tol[lo:hi]).all()
        if what != "page":
            assert (got[b.cu[1]:b.cu[2]] == 7.0).all()
    cu = i32([0, 2, 4, 6, 9])                            # past the token array
    out.fill_(7.0)
    mla.mla_attn_paged(d["q_lat"], d["q_pe"], d["pages"], d["block_table"], cu, d["seq_len"], out, scale=SCALE)
    assert mla.mla_get_device_error() == INVALID
    assert (out[6:] == 7.0).all() and torch.isfinite(out[:6]).all() and (out[:6] != 7.0).any()
    table = d["block_table"].clone()
    table[0, 0] = -1
    rows = torch.full((4, 576), 7.0, dtype=torch.float16, device="cuda")
    mla.mla_paged_gather(d["pages"], table, i32([14, 0, 0, b.width * 16 - 1]), i32([0, 4, 4, 4, 4]), rows)
    assert mla.mla_get_device_error() == INVALID         # rows 14, 15 are on the bad page
    assert (rows[:2] == 7.0).all() and (rows[2:] != 7.0).any()
    mla.mla_paged_gather(d["pages"], d["block_table"], i32([0, 0, 0, b.width * 16 - 1]), i32([0, 0, 0, 0, 2]), rows)
    assert mla.mla_get_device_error() == INVALID


@pytest.mark.parametrize("e4m3", [False, True])
@pytest.mark.parametrize("cu,whole", [([0, 4, 8, 13], 8), ([0, 4, 40, 40], 4), ([0, 8, 4, 12], 0), ([-2, 4, 8, 12], 0),
                                      ([12, 12, 12, 12], 0), ([0, 4, 8, 12], 12)], ids=str)
def test_read_back_reports_rows_outside_the_output(cu, whole, e4m3):
    """`whole`: rows of the output in front that the call defines, whatever it reports."""
    b = Batch(27, e4m3, 16, 16, [40, 33, 20], [40, 33, 20])
    d = b.dev()
    out = torch.full((12, 576), 7.0, dtype=torch.float16, device="cuda")
    mla.mla_paged_gather(d["pages"], d["block_table"], None, i32(cu), out)
    torch.cuda.synchronize()
    good = cu[0] >= 0 and all(x <= y for x, y in zip(cu, cu[1:])) and cu[-1] <= 12
    assert mla.mla_get_device_error() == (0 if good else INVALID)
    want = np.concatenate([b.rows[s][:max(0, cu[s + 1] - cu[s])] for s in range(3)]) if whole else np.zeros((0, 576))
    assert np.array_equal(out[:whole].double().cpu().numpy(), want[:whole])


# ---------------------------------------------------------------------------
# attention
# ---------------------------------------------------------------------------
SHAPES = [                                               # heads, page, news, lens
    (16, 16, [1], [1]), (16, 64, [1], [64]), (128, 64, [1], [65]), (48, 32, [1], [1000]),
    (128, 16, [1, 1, 1], [17, 300, 2049]), (16, 64, [5], [5]), (16, 128, [64, 1, 0, 7], [64, 63, 9, 200]),
    (80, 16, [33, 2], [40, 129]), (112, 64, [9, 1], [700, 513]), (32, 256, [130], [301]),
]


@pytest.mark.parametrize("e4m3", [False, True])
@pytest.mark.parametrize("shape", SHAPES, ids=str)
def test_attention_over_pages(shape, e4m3):
    H, ps, news, lens = shape
    b = Batch(11, e4m3, H, ps, news, lens, pad=2)
    check(b, run(b))


@pytest.mark.parametrize("e4m3", [False, True])
@pytest.mark.parametrize("window,n_sink", [(1, 0), (1, 1), (63, 0), (64, 4), (65, 64), (200, 70), (128, 1000)])
def test_attention_in_a_window_with_sinks(window, n_sink, e4m3):
    b = Batch(12, e4m3, 16, 16, [1, 40, 3, 0, 130], [500, 333, 3, 20, 701], window, n_sink)
    check(b, run(b))
    b = Batch(13, e4m3, 128, 64, [1, 2], [1000, 450], window, n_sink)
    check(b, run(b))


@pytest.mark.parametrize("e4m3", [False, True])
def test_attention_split_over_the_keys(e4m3):
    b = Batch(14, e4m3, 16, 64, [1, 12], [20000, 9999])
    check(b, run(b))
    b = Batch(15, e4m3, 64, 16, [3], [12345], 6000, 20)
    check(b, run(b))


@pytest.mark.parametrize("e4m3", [False, True])
@pytest.mark.parametrize("B,H,top", [(5, 128, 128), (24, 16, 900), (30, 128, 500), (90, 128, 200), (700, 16, 90)])
def test_batches_from_few_blocks_to_many(B, H, top, e4m3):
    """Blocks that are not cut, equal shares, a run shared by all clusters, more sequences than threads; some
    sequences bring two tokens, some none."""
    rng = np.random.default_rng(B)
    news = [int(n) for n in rng.choice((0, 1, 1, 1, 1, 2), B)]
    lens = [max(n, int(x)) for n, x in zip(news, rng.integers(1, top + 1, B))]
    news[0], lens[0] = 1, top
    b = Batch(22, e4m3, H, 16, news, lens, pad=3)
    check(b, run(b))


@pytest.mark.parametrize("e4m3", [False, True])
@pytest.mark.parametrize("H,news", [(16, [1, 8, 0, 0, 0, 0, 0, 0, 0, 1]), (48, [4, 0, 1, 0, 0, 0]), (112, [1, 2, 1, 0]),
                                    (80, [1] * 100), (32, [0, 3, 0, 1])], ids=str)
def test_blocks_of_few_rows_beside_full_ones(H, news, e4m3):
    """No more tokens than sequences, few heads: warps without rows, blocks of one and of all rows in turn."""
    lens = [50 + 97 * (i * 7 % 10) for i in range(len(news))]
    b = Batch(23, e4m3, H, 64, news, lens, pad=1)
    b.T = min(b.T, len(news))                            # at most a token per sequence in the token array
    b.q_lat, b.q_pe = b.q_lat[:b.T], b.q_pe[:b.T]
    check(b, run(b))


@pytest.mark.parametrize("H", [16, 48, 112])
def test_queries_of_few_rows_follow_one_another(H):
    """Several pieces a cluster, single tokens of few heads: warps that read no scores write the next queries."""
    rng = np.random.default_rng(H)
    lens = [int(x) for x in rng.integers(1, 200, 500)]
    b = Batch(25, False, H, 16, [1] * len(lens), lens)
    check(b, run(b))


@pytest.mark.parametrize("top", [64, 300])
def test_many_short_blocks_in_the_e4m3_ring(top):
    """Several pieces a cluster, of one tile each or of one to five: their queries and tiles follow one another
    through the ring's stages (test_paged_ring.py has the order in which stages are released)."""
    rng = np.random.default_rng(top)
    lens = [int(x) for x in rng.integers(1, top + 1, 500)]
    b = Batch(24, True, 128, 16, [1] * len(lens), lens)
    check(b, run(b))


@pytest.mark.parametrize("news", [[100, 128, 100], [160, 200, 160]], ids=str)
def test_e4m3_chunks_beyond_the_staging(news):
    """Chunks of too few blocks to be staged; two that are staged and a third that no longer fits.  On a few pages
    named many times."""
    ps, H, lens = 64, 16, [70001, 50000, 30001]
    rng = np.random.default_rng(8)
    raw = PO.pack_rows(bf16(rng.standard_normal((8 * ps, 512))), bf16(rng.standard_normal((8 * ps, 64))), True)
    pages = torch.from_numpy(raw).cuda().reshape(8, ps, 656)
    vals = torch.from_numpy(PO.row_values(raw, True)).cuda()
    table = torch.from_numpy(rng.integers(0, 8, (3, -(-max(lens) // ps))).astype(np.int32)).cuda()
    T = sum(news)
    q_lat = torch.from_numpy(rng.standard_normal((T, H, 512)).astype(np.float16)).cuda()
    q_pe = torch.from_numpy(bf16(rng.standard_normal((T, H, 64)))).bfloat16().cuda()
    out = torch.full((T, H, 512), float("nan"), dtype=torch.float16, device="cuda")
    mla.mla_attn_paged(q_lat, q_pe, pages, table, i32(np.concatenate([[0], np.cumsum(news)])), i32(lens), out,
                       scale=SCALE)
    torch.cuda.synchronize()
    assert mla.mla_get_device_error() == 0
    at = 0
    for b in range(3):
        p = torch.arange(lens[b], device="cuda")
        rows = vals[table[b].long()[p // ps] * ps + p % ps]
        for i in (0, news[b] - 1):
            n = lens[b] - news[b] + i + 1
            q = torch.cat([q_lat[at + i].double(), q_pe[at + i].double()], -1)
            w = ((q @ rows[:n].T) * SCALE).softmax(-1)
            ref, mag = w @ rows[:n, :512], w @ rows[:n, :512].abs()
            tol = (2.0 ** -11 + 2.0 ** -12) * mag + 2.0 ** -11 * ref.abs() + 2.0 ** -24
            assert ((out[at + i].double() - ref).abs() <= tol).all()
        at += news[b]


def test_a_chunk_of_more_than_2_to_the_24_tiles():
    """8600 tokens of 128 heads at the end of 131500 rows, on a few pages named many times."""
    ps, H, T, L = 64, 128, 8600, 131500
    g = torch.Generator(device="cuda").manual_seed(9)
    pages = torch.randn(8, ps, 576, device="cuda", generator=g).half()
    table = torch.randint(0, 8, (1, -(-L // ps)), dtype=torch.int32, device="cuda", generator=g)
    q_lat = torch.randn(T, H, 512, device="cuda", generator=g, dtype=torch.float16)
    q_pe = torch.randn(T, H, 64, device="cuda", generator=g, dtype=torch.bfloat16)
    out = torch.full((T, H, 512), float("nan"), dtype=torch.float16, device="cuda")
    mla.mla_attn_paged(q_lat, q_pe, pages, table, i32([0, T]), i32([L]), out, scale=SCALE)
    torch.cuda.synchronize()
    assert mla.mla_get_device_error() == 0
    assert torch.isfinite(out).all()
    p = torch.arange(L, device="cuda")
    rows = pages.reshape(-1, 576)[table[0].long()[p // ps] * ps + p % ps].double()
    for i in (0, 4321, T - 1):
        n = L - T + i + 1
        w = ((torch.cat([q_lat[i].double(), q_pe[i].double()], -1) @ rows[:n].T) * SCALE).softmax(-1)
        ref, mag = w @ rows[:n, :512], w @ rows[:n, :512].abs()
        tol = (2.0 ** -11 + 2.0 ** -12) * mag + 2.0 ** -11 * ref.abs() + 2.0 ** -24
        assert ((out[i].double() - ref).abs() <= tol).all()


def test_a_block_that_takes_longer_than_a_wait_may():
    """80 sequences of 45 million rows, on two pages named many times: a cluster works on one block for more than half
    a second, the limit of a wait.  All keys behind the first page score 200 below, so the output is the first
    page's."""
    ps, n, B, H = 4096, 11000, 80, 16
    g = torch.Generator(device="cuda").manual_seed(12)
    pages = torch.randn(2, ps, 576, device="cuda", generator=g).half()
    pages[:, :, 512:] = 0
    pages[1, :, 512] = -200.0
    table = torch.ones(B, n, dtype=torch.int32, device="cuda")
    table[:, 0] = 0
    q_lat = torch.randn(B, H, 512, device="cuda", generator=g, dtype=torch.float16)
    q_pe = torch.zeros(B, H, 64, device="cuda", dtype=torch.bfloat16)
    q_pe[:, :, 0] = 16.0                                 # x 200 x 0.072 = 231, below every score of the first page
    out = torch.full((B, H, 512), float("nan"), dtype=torch.float16, device="cuda")
    mla.mla_attn_paged(q_lat, q_pe, pages, table, i32(np.arange(B + 1)), i32([n * ps - 37] * B), out, scale=SCALE)
    torch.cuda.synchronize()
    assert mla.mla_get_device_error() == 0
    rows = pages[0, :, :512].double()
    w = ((q_lat.double() @ rows.T) * SCALE).softmax(-1)
    ref, mag = w @ rows, w @ rows.abs()
    tol = (2.0 ** -11 + 2.0 ** -12) * mag + 2.0 ** -11 * ref.abs() + 2.0 ** -24 + 2.0 ** -25 * ps * rows.abs().max()
    assert ((out.double() - ref).abs() <= tol).all()


def test_sharp_and_flat_scores():
    # nearly one key for each row; all keys alike (their mean); and all rows the same row
    for kw in (dict(std=6.0), dict(std=1e-3), dict(same=True)):
        b = Batch(16, False, 16, 64, [3, 1], [500, 1000], **kw)
        if "std" in kw and kw["std"] > 1:
            # scores reach ~60 in magnitude: fp32 sums of them move a probability by 2^-10 more
            torch.cuda.synchronize()
            ref, tol = b.ref()
            got = run(b).float().cpu().numpy()
            assert (np.abs(got - ref) <= 2 * tol).all()
        else:
            check(b, run(b))


def test_strided_table_offsets_and_order_of_the_batch():
    b = Batch(17, False, 32, 16, [4, 1, 20], [100, 77, 20])
    d = b.dev()
    wide = torch.full((b.B, b.width + 9), -7, dtype=torch.int32, device="cuda")
    wide[:, :b.width] = d["block_table"]
    want = run(b, d)
    check(b, want)
    d["block_table"] = wide[:, :b.width]
    assert torch.equal(torch.nan_to_num(run(b, d)), torch.nan_to_num(want))
    # two sequences on the same pages (a shared prefix)
    d["block_table"] = d["block_table"][[0, 0, 2]].contiguous()
    d["seq_len"][1] = 97
    out = run(b, d)
    ref, _, _ = PO.attend(np.concatenate([b.q_lat[4:5], b.q_pe[4:5]], -1).astype(np.float64), b.rows[0][:97], 96, 0, 0,
                          SCALE)
    assert np.abs(out[4].float().cpu().numpy() - ref[0]).max() <= 2.0 ** -9 * np.abs(ref).max()
    assert mla.mla_get_device_error() == 0


@pytest.mark.parametrize("e4m3", [False, True])
def test_rows_behind_the_32_bit_offsets(e4m3):
    """Pages whose rows lie more than 4 GiB into the pool: written, attended over and read back."""
    b = Batch(20, e4m3, 16, 64, [3, 70], [200, 90])
    d, extra = b.dev(), 60000 if not e4m3 else 105000
    pages = torch.empty(extra + b.n_pages, 64, d["pages"].shape[2], dtype=d["pages"].dtype, device="cuda")
    pages[:3].view(torch.uint8).fill_(0xFF)              # what a wrapped offset would read: NaN
    pages[extra:] = d["pages"]
    assert pages[extra:].data_ptr() - pages.data_ptr() > 1 << 32
    d["pages"] = pages
    d["block_table"] = torch.where((d["block_table"] >= 0) & (d["block_table"] < b.n_pages), d["block_table"] + extra,
                                   d["block_table"])
    check(b, run(b, d))
    out = torch.empty(200, 576, dtype=torch.float16, device="cuda")
    mla.mla_paged_gather(pages, d["block_table"][:1].contiguous(), None, i32([0, 200]), out)
    assert np.array_equal(out.double().cpu().numpy(), b.rows[0])
    c = torch.full((1, 512), 3.0, dtype=torch.bfloat16, device="cuda")
    k = torch.zeros(1, 64, dtype=torch.bfloat16, device="cuda")
    mla.mla_paged_append(c, k, pages, d["block_table"][:1].contiguous(), i32([0, 1]), i32([150]))
    mla.mla_paged_gather(pages, d["block_table"][:1].contiguous(), i32([149]), i32([0, 1]), out)
    assert (out[0, :512] == 3).all() and (out[0, 512:] == 0).all()
    assert mla.mla_get_device_error() == 0


def test_a_decreasing_cu_is_reported_and_stays_in_bounds():
    b = Batch(21, False, 16, 16, [4, 4, 4], [40, 30, 20])
    d = b.dev()
    d["cu_q"] = i32([0, 8, 2, 12])
    out = run(b, d)
    torch.cuda.synchronize()
    assert mla.mla_get_device_error() == INVALID
    assert run(b).isfinite().all()                       # the next call is not affected
    assert mla.mla_get_device_error() == 0


@pytest.mark.parametrize("cu,lens", [
    ([0, 23, 24, 21, 54, 13, 21, 60], [76, 163070, 119811, 60, 8312, 1783, 84]),
    ([0, 13, 17, 13, 20, 8, 17, 9, 12, 11, 20], [682, 172736, 1706, 199, 814, 2440, 2384, 1866, 52, 40]),
    ([0, 16, 2, 16, 5, 1, 9, 20, 20], [186009, 1445, 409, 94, 68, 1518, 795, 2423])], ids=str)
def test_a_decreasing_cu_with_blocks_behind_the_total(cu, lens):
    """Offsets with which the walk over the blocks meets long ones that the total does not count: a block's end then
    lies up to eight times the total away, and the merge must not look for partials there."""
    T, H = cu[-1], 128
    g = torch.Generator(device="cuda").manual_seed(10)
    pages = torch.randn(4, 64, 576, device="cuda", generator=g).half()
    table = torch.randint(0, 4, (len(lens), -(-max(lens) // 64)), dtype=torch.int32, device="cuda", generator=g)
    q_lat = torch.randn(T, H, 512, device="cuda", generator=g, dtype=torch.float16)
    q_pe = torch.randn(T, H, 64, device="cuda", generator=g, dtype=torch.bfloat16)
    out = torch.zeros(T, H, 512, dtype=torch.float16, device="cuda")
    mla.mla_attn_paged(q_lat, q_pe, pages, table, i32(cu), i32(lens), out, scale=SCALE)
    torch.cuda.synchronize()
    assert mla.mla_get_device_error() == INVALID
    b = Batch(21, False, 16, 16, [4, 4, 4], [40, 30, 20])
    check(b, run(b))


@pytest.mark.parametrize("H", [16, 128])
@pytest.mark.parametrize("where", ["first", "last"])
@pytest.mark.parametrize("gap", [8.0, 14.0, 16.0, 18.0])
def test_a_leading_key_of_small_values(gap, where, H):
    """One key, with values of zero, whose score leads all 98304 others by `gap` (an attention sink): the output is the
    others' small share.  As many sequences as leave their blocks whole."""
    ps, L, B = 64, 98305, 152
    g = torch.Generator(device="cuda").manual_seed(13)
    pages = (torch.randn(-(-L // ps), ps, 576, device="cuda", generator=g) + 1.0).half()
    pages[:, :, 512:] = 0
    lead = 0 if where == "first" else L - 1
    pages.view(-1, 576)[lead] = 0
    pages.view(-1, 576)[lead, 512] = 1.0
    table = torch.arange(len(pages), dtype=torch.int32, device="cuda").repeat(B, 1)
    q_lat = torch.zeros(B, H, 512, dtype=torch.float16, device="cuda")
    q_pe = torch.zeros(B, H, 64, dtype=torch.bfloat16, device="cuda")
    q_pe[:, :, 0] = 128.0
    scale = gap / 128.0                                  # exact: scores of 0 and of gap
    out = torch.full((B, H, 512), float("nan"), dtype=torch.float16, device="cuda")
    mla.mla_attn_paged(q_lat, q_pe, pages, table, i32(np.arange(B + 1)), i32([L] * B), out, scale=scale)
    torch.cuda.synchronize()
    assert mla.mla_get_device_error() == 0
    rows = pages.view(-1, 576)[:L, :512].double()
    w = float(np.exp(-gap))
    total = 1.0 + (L - 1) * w
    ref, mag = rows.sum(0) * w / total, rows.abs().sum(0) * w / total
    # P to fp16: 2^-11 of itself, or below fp16's normal range 2^-25 where the largest is 2^7 at least; its exponent
    # in fp32 (three roundings at up to 33, the exponential's own 2^-22): 2^-18; sums in fp32 of 16 products a step, a
    # last place each; row sums in fp32, half of one a tile; the output to fp16
    tol = ((2.0 ** -11 + 2.0 ** -18 + L / 16 * 2.0 ** -23) * mag + 2.0 ** -32 * L * rows.abs().mean(0)
           + (2.0 ** -11 + (L / 64 + 1) * 2.0 ** -24) * ref.abs() + 2.0 ** -25)
    off = ((out.double() - ref).abs() / tol).max().item()
    assert off <= 1.0, off


@pytest.mark.parametrize("e4m3", [False, True])
@pytest.mark.parametrize("H,L", [(16, 66), (128, 200), (64, 20000)])
def test_weights_sum_to_one(H, L, e4m3):
    """Rows of equal latents with different RoPE keys: whatever the weights, the output is that latent, to the bit (the
    sums' fp32 roundings are far below half an fp16 step).  The first key scores 0, one of the second tile 2^7 (1 +
    0.98 x 2^-11) times as much: less than lets the running maximum move, and almost half a step from an fp16 value, so
    that the output would be 1.8 half steps off if the row sum did not have the same rounding."""
    ps = 64
    lat = torch.full((-(-L // ps) * ps, 512), 1.875)
    rope = torch.zeros(len(lat), 64)
    rope[1:, 0] = -1000.0
    rope[65, 0] = 100.0
    raw = torch.from_numpy(PO.pack_rows(lat.numpy(), rope.numpy(), e4m3)).cuda()
    pages = (raw if e4m3 else raw.view(torch.float16)).reshape(len(lat) // ps, ps, -1)
    table = torch.arange(len(pages), dtype=torch.int32, device="cuda")[None]
    q_lat = torch.zeros(1, H, 512, dtype=torch.float16, device="cuda")
    q_pe = torch.zeros(1, H, 64, dtype=torch.bfloat16, device="cuda")
    q_pe[:, :, 0] = 1.0
    scale = (7.0 + np.log2(1.0 + 0.98 * 2.0 ** -11)) / 100.0 * np.log(2.0)
    out = torch.full((1, H, 512), float("nan"), dtype=torch.float16, device="cuda")
    mla.mla_attn_paged(q_lat, q_pe, pages, table, i32([0, 1]), i32([L]), out, scale=scale)
    torch.cuda.synchronize()
    assert mla.mla_get_device_error() == 0
    assert (out == 1.875).all()


@pytest.mark.parametrize("e4m3", [False, True])
def test_calls_behind_a_recorded_timeout_end_and_leave_the_next_one_right(e4m3):
    """While the error word holds a timeout, waits that do not complete at once give up: every role of the kernel then
    leaves early, with loads and products under way."""
    few, many = Batch(28, e4m3, 16, 16, [1, 5], [300, 90]), Batch(29, e4m3, 128, 64, [1] * 90, [777] * 90)
    d = [(b, b.dev()) for b in (few, many)]
    mla.mla_selftest_wait_timeout(1000)
    for b, x in d:
        run(b, x)                                        # undefined outputs
    assert mla.mla_get_device_error() == -6
    for b, x in d:
        check(b, run(b, x))


@pytest.mark.parametrize("e4m3", [False, True])
@pytest.mark.parametrize("B,H,lead", [(152, 128, 15), (152, 16, 16), (152, 16, 17), (20, 48, 100), (3, 128, 16)])
def test_sums_over_a_million_rows(B, H, lead, e4m3):
    """Values of one sign, over rows that all count, in whole blocks (152 sequences), in blocks that are cut, and with
    one page whose scores move the running maximum around the place (65536 rows) where sums are moved on."""
    ps, L = 4096, (1 << 20) - 77
    rng = np.random.default_rng(15)
    lat, rope = np.zeros((8 * ps, 512), np.float32), np.zeros((8 * ps, 64), np.float32)
    lat[:] = bf16(rng.uniform(1.0, 2.0, lat.shape))
    rope[7 * ps:, 0] = 1.0                               # the leading page
    raw = torch.from_numpy(PO.pack_rows(lat, rope, e4m3)).cuda()
    pages = (raw if e4m3 else raw.view(torch.float16)).reshape(8, ps, -1)
    table = rng.integers(0, 7, (1, 256))
    table[0, lead] = 7
    q_lat = torch.zeros(B, H, 512, dtype=torch.float16, device="cuda")
    q_pe = torch.zeros(B, H, 64, dtype=torch.bfloat16, device="cuda")
    q_pe[:, :, 0] = 1.0
    gap = 5.875                                          # 8.5 in log2: the running maximum moves
    out = torch.full((B, H, 512), float("nan"), dtype=torch.float16, device="cuda")
    mla.mla_attn_paged(q_lat, q_pe, pages, i32(np.repeat(table, B, 0)), i32(np.arange(B + 1)), i32([L] * B), out,
                       scale=gap)
    torch.cuda.synchronize()
    assert mla.mla_get_device_error() == 0
    rows = PO.row_values(raw.cpu().numpy(), e4m3)[:, :512].reshape(8, ps, 512)
    n = np.full(256, ps)
    n[-1] = L - 255 * ps
    w = np.where(table[0] == 7, np.exp(gap), 1.0)
    total = (w * n).sum()
    ref = sum(w[i] * rows[table[0, i], :n[i]].sum(0) for i in range(256)) / total
    # relative, all values being positive: P to fp16 and the output to fp16 2^-11 each; the products' sums a last place
    # (2^-23) for each 16 keys of 65536 rows, 2^-11; the row sum half of one a tile, 16384 x 2^-24; the exponent 2^-18
    tol = 3 * 2.0 ** -11 + 2.0 ** -10 + 2.0 ** -18
    off = np.abs(out.double().cpu().numpy() / ref - 1.0).max()
    assert off <= tol, f"{off:.2e} of {tol:.2e}"


@pytest.mark.parametrize("e4m3", [False, True])
def test_same_call_same_bits_on_two_streams(e4m3):
    b = Batch(18, e4m3, 128, 64, [1, 1, 5], [3000, 5000, 900])
    d = b.dev()
    first = run(b, d)
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in range(2)]
    outs = []
    for s in streams:                                    # two calls at once, a workspace each
        with torch.cuda.stream(s):
            outs.append(run(b, d))
    torch.cuda.synchronize()
    for o in outs:
        assert torch.equal(o, first)
    explicit = torch.empty_like(first)
    run(b, d, explicit, stream=streams[0])
    torch.cuda.synchronize()
    assert torch.equal(explicit, first)
    check(b, first)


@pytest.mark.parametrize("e4m3", [False, True])
def test_captured_step_follows_its_arrays(e4m3):
    """One captured step (append, absorb, attention, decompression) replayed while sequences grow and swap."""
    rng = np.random.default_rng(6)
    H, ps, n_pages, B, T = 16, 16, 64, 3, 24
    dev = lambda x: torch.from_numpy(np.asarray(x, np.float32)).bfloat16().cuda()    # noqa: E731
    wk, wv = (bf16(rng.standard_normal((H, 128, 512)) / np.sqrt(128)), bf16(rng.standard_normal((H, 512, 128)) / np.sqrt(512)))
    x = dict(q_nope=torch.zeros(T, H, 128, dtype=torch.bfloat16, device="cuda"),
             q_pe=torch.zeros(T, H, 64, dtype=torch.bfloat16, device="cuda"),
             c_kv=torch.zeros(T, 512, dtype=torch.bfloat16, device="cuda"),
             k_pe=torch.zeros(T, 64, dtype=torch.bfloat16, device="cuda"))
    cu, lens = i32([0, 20, 21, 24]), i32([20, 1, 3])
    order = rng.permutation(n_pages).astype(np.int32)
    table = torch.from_numpy(order[:60].reshape(3, 20).copy()).cuda()
    pages = P.paged_pages(n_pages, ps, e4m3)
    pages.zero_()
    bufs = P.paged_buffers(T, H)
    wkd, wvd = dev(wk), dev(wv)

    def step():
        P.mla_paged_step(x["q_nope"], x["q_pe"], x["c_kv"], x["k_pe"], wkd, wvd, pages, table, cu, lens, bufs=bufs,
                         window=25, n_sink=2)

    step()
    torch.cuda.synchronize()
    g, s = torch.cuda.CUDAGraph(), torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.graph(g, stream=s):
        step()
    length, rows = [0, 0, 0], [np.zeros((0, 576)) for _ in range(3)]
    for news in ([20, 1, 3], [1, 20, 0], [1, 1, 1], [3, 5, 16], [0, 0, 24]):
        new = {k: bf16(rng.standard_normal(v.shape)) for k, v in x.items()}
        for k in x:
            x[k].copy_(dev(new[k]))
        cun = np.concatenate([[0], np.cumsum(news)])
        cu.copy_(i32(cun))
        length = [l + n for l, n in zip(length, news)]
        lens.copy_(i32(length))
        g.replay()
        torch.cuda.synchronize()
        assert mla.mla_get_device_error() == 0
        got = bufs.o.cpu().numpy()
        for b in range(3):
            lo, hi = cun[b], cun[b + 1]
            pos = np.arange(length[b] - news[b], length[b])
            raw = PO.pack_rows(new["c_kv"][lo:hi], PO.rope_rows(new["k_pe"][lo:hi], pos, FB, FS), e4m3)
            rows[b] = np.concatenate([rows[b], PO.row_values(raw, e4m3)])
            if news[b] == 0:
                continue
            ql = O.absorb_q(new["q_nope"][lo:hi], wk)
            ol, _, _ = PO.attend(np.concatenate([ql, new["q_pe"][lo:hi]], -1).astype(np.float64), rows[b],
                                 int(pos[0]), 25, 2, SCALE)
            ref = O.late_decompress(ol, wv)
            d = np.abs(got[lo:hi] - ref)
            # q_lat, the probabilities and o_lat are rounded to fp16 on the way: 1e-3 in the mean
            assert d.mean() <= 1.5e-3 * np.abs(ref).mean() and d.max() <= 1e-2 * np.abs(ref).max()
        if cun[-1] == 2:
            assert np.isfinite(got).all()


@pytest.mark.parametrize("stream", [0, 1])
def test_a_step_on_the_default_stream_by_its_handle(stream, monkeypatch):
    """Its buffers come from that stream, and so does the zero fill of o_lat."""
    H, seen = 16, []
    make = P.paged_buffers
    monkeypatch.setattr(P, "paged_buffers", lambda *a: (seen.append(torch.cuda.current_stream()), make(*a))[1])
    g = torch.Generator(device="cuda").manual_seed(14)
    bf = lambda *s: torch.randn(*s, generator=g, device="cuda").bfloat16()             # noqa: E731
    args = (bf(2, H, 128), bf(2, H, 64), bf(2, 512), bf(2, 64), bf(H, 128, 512), bf(H, 512, 128) / 22)
    table, cu, lens = torch.tensor([[0]], dtype=torch.int32, device="cuda"), i32([0, 2]), i32([2])
    outs = []
    for s in (None, stream):
        pages = P.paged_pages(1, 16)
        outs.append(P.mla_paged_step(*args, pages, table, cu, lens, stream=s).o.clone())
    torch.cuda.synchronize()
    assert mla.mla_get_device_error() == 0
    assert seen == [torch.cuda.default_stream()] * 2
    assert torch.equal(*outs) and outs[0].abs().max() > 0


def test_read_back_feeds_the_flat_prefill():
    """A prefix in pages, read back as flat rows, gives the flat prefill the same answer as the pages give."""
    b = Batch(19, False, 16, 64, [40], [200])
    d = b.dev()
    flat = torch.empty(200, 576, dtype=torch.bfloat16, device="cuda")
    mla.mla_paged_gather(d["pages"], d["block_table"], None, i32([0, 200]), flat)
    o = torch.empty(40, 16, 512, dtype=torch.float16, device="cuda")
    mla.mla_attn_prefill(d["q_lat"], d["q_pe"], flat, 160, o, scale=SCALE)
    p = run(b, d)
    torch.cuda.synchronize()
    assert mla.mla_get_device_error() == 0
    a, c = o.float(), p.float()
    assert (a - c).abs().mean() <= 2e-3 * c.abs().mean() and (a - c).abs().max() <= 1e-2 * c.abs().max()
