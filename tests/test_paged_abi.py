"""Refusals of the paged entry points, on the host (no GPU needed), and the oracle's row formats."""
import ctypes

import numpy as np
import pytest
import torch

import mla_latent_kv_lat_gb300 as mla
from mla_latent_kv_lat_gb300 import binding, build, pipeline
from oracle import paged_oracle as PO
from tests.paged_util import Batch

P = ctypes.c_void_p
GOOD, OUT, ODD, ODD4 = 0x100000, 0x90000000, 0x100008, 0x100002   # never dereferenced: the checks fail first


@pytest.fixture(scope="module")
def lib():
    build.build()
    return mla.load_library()


def cache(**kw):
    c = binding.MLAPagedCache(GOOD, GOOD, 8, 8, 100, 64, 0)
    for k, v in kw.items():
        setattr(c, k, v)
    return ctypes.byref(c)


BAD_CACHES = [(dict(pages=None), -1), (dict(pages=ODD), -3), (dict(block_table=None), -1), (dict(block_table=ODD4), -3),
              (dict(table_stride=7), -1), (dict(table_stride=-1), -1), (dict(max_pages=0), -1), (dict(n_pages=0), -1),
              (dict(page_size=8), -2), (dict(page_size=48), -2), (dict(page_size=8192), -2), (dict(type=2), -2),
              (dict(type=-1), -2), (dict(n_pages=1 << 26, page_size=64), -2)]


def test_bad_caches_are_refused(lib):
    d = ctypes.byref(binding.make_dims(16))
    ws = lib.mla_paged_workspace_size(d)
    assert ws > 0
    for kw, want in BAD_CACHES:
        assert lib.mla_paged_append(cache(**kw), GOOD, GOOD, GOOD, GOOD, 2, 4, 1e4, 1.0, None) == want, kw
        assert lib.mla_paged_gather(cache(**kw), None, GOOD, 2, 4, GOOD, 0, None) == want, kw
        assert lib.mla_attn_paged(d, GOOD, GOOD, cache(**kw), GOOD, GOOD, 2, 4, 0, 0, GOOD, ws, OUT, None) == want, kw
    assert lib.mla_paged_append(None, GOOD, GOOD, GOOD, GOOD, 2, 4, 1e4, 1.0, None) == -1


def test_bad_arguments_are_refused(lib):
    ap, ga, at = lib.mla_paged_append, lib.mla_paged_gather, lib.mla_attn_paged
    for a in ((None, GOOD, GOOD, GOOD, 2, 4, 1e4, 1.0), (GOOD, GOOD, None, GOOD, 2, 4, 1e4, 1.0),
              (GOOD, GOOD, GOOD, None, 2, 4, 1e4, 1.0), (GOOD, GOOD, GOOD, GOOD, 0, 4, 1e4, 1.0),
              (GOOD, GOOD, GOOD, GOOD, 2, 0, 1e4, 1.0), (GOOD, GOOD, GOOD, GOOD, 2, 4, 1.0, 1.0),
              (GOOD, GOOD, GOOD, GOOD, 2, 4, 1e4, float("nan"))):
        assert ap(cache(), *a, None) == -1
    assert ap(cache(), ODD, GOOD, GOOD, GOOD, 2, 4, 1e4, 1.0, None) == -3
    assert ap(cache(), GOOD, GOOD, ODD4, GOOD, 2, 4, 1e4, 1.0, None) == -3
    assert ap(cache(table_stride=70000, max_pages=1), GOOD, GOOD, GOOD, GOOD, 65536, 4, 1e4, 1.0, None) == -2
    assert ga(cache(), None, None, 2, 4, GOOD, 0, None) == -1
    assert ga(cache(), ODD4, GOOD, 2, 4, GOOD, 0, None) == -3
    assert ga(cache(), None, GOOD, 2, 4, ODD, 0, None) == -3
    assert ga(cache(), None, GOOD, 2, 0, GOOD, 0, None) == -1
    d = ctypes.byref(binding.make_dims(16))
    ws = lib.mla_paged_workspace_size(d)
    assert at(d, GOOD, GOOD, cache(), GOOD, GOOD, 2, 4, -1, 0, GOOD, ws, OUT, None) == -1
    assert at(d, GOOD, GOOD, cache(), GOOD, GOOD, 2, 4, 8, -1, GOOD, ws, OUT, None) == -1
    assert at(d, GOOD, GOOD, cache(), GOOD, GOOD, 2, 0, 0, 0, GOOD, ws, OUT, None) == -1
    assert at(d, GOOD, GOOD, cache(), GOOD, GOOD, 0, 4, 0, 0, GOOD, ws, OUT, None) == -1
    assert at(d, GOOD, None, cache(), GOOD, GOOD, 2, 4, 0, 0, GOOD, ws, OUT, None) == -1
    assert at(d, GOOD, GOOD, cache(), GOOD, GOOD, 2, 4, 0, 0, None, ws, OUT, None) == -4
    assert at(d, GOOD, GOOD, cache(), GOOD, GOOD, 2, 4, 0, 0, GOOD, ws - 1, OUT, None) == -4
    assert at(d, GOOD, GOOD, cache(), GOOD, GOOD, 2, 4, 0, 0, ODD, ws, OUT, None) == -3
    assert at(d, GOOD, GOOD, cache(), GOOD, GOOD, 2, 1 << 28, 0, 0, GOOD, ws, OUT, None) == -2
    # q_lat and o_lat (4 tokens x 16 heads x 1024 bytes) must not overlap
    for o in (GOOD, GOOD + 65536 - 16, GOOD - 65536 + 16):
        assert at(d, GOOD, GOOD, cache(), GOOD, GOOD, 2, 4, 0, 0, GOOD, ws, o, None) == -1
    bad = binding.make_dims(24)
    assert at(ctypes.byref(bad), GOOD, GOOD, cache(), GOOD, GOOD, 2, 4, 0, 0, GOOD, ws, OUT, None) == -2
    assert lib.mla_paged_workspace_size(ctypes.byref(bad)) == 0


def test_overlapping_memory_is_refused(lib):
    """What a call writes, laid over the first and the last 16 (or 4) bytes of each thing that it reads."""
    B, T, H, far = 3, 5, 16, 0x400000000
    d = ctypes.byref(binding.make_dims(H))
    ws = lib.mla_paged_workspace_size(d)
    for type_, row in ((0, 1152), (1, 656)):
        pool, table = 100 * 64 * row, ((B - 1) * 9 + 8) * 4
        # every span at a place of its own, 4 GB apart
        sizes = dict(pages=pool, table=table, cu=4 * (B + 1), len=4 * B, a=T * 1024, b=T * 128, ql=T * H * 1024,
                     qp=T * H * 128, o=T * H * 1024, ws=ws, out=T * 1152, row0=4 * B)
        place = {k: far * (i + 1) for i, k in enumerate(sizes)}

        def calls(at):
            c = cache(pages=at["pages"], block_table=at["table"], table_stride=9, type=type_)
            return dict(
                append=lambda: lib.mla_paged_append(c, at["a"], at["b"], at["cu"], at["len"], B, T, 1e4, 1.0, None),
                gather=lambda: lib.mla_paged_gather(c, at["row0"], at["cu"], B, T, at["out"], 0, None),
                attn=lambda: lib.mla_attn_paged(d, at["ql"], at["qp"], c, at["cu"], at["len"], B, T, 0, 0, at["ws"], ws,
                                                at["o"], None))
        reads = dict(append=("a", "b", "table", "cu", "len"), gather=("pages", "table", "cu", "row0"),
                     attn=("ql", "qp", "pages", "table", "cu", "len"))
        writes = dict(append=("pages",), gather=("out",), attn=("o", "ws"))
        for call in reads:
            for w in writes[call]:
                for r in reads[call] + tuple(x for x in writes[call] if x != w):
                    first, last = place[r] - sizes[w] + 16, place[r] + (sizes[r] - 1) // 16 * 16
                    for to in (first + (-first) % 16, last):
                        assert calls(dict(place, **{w: to}))[call]() == -1, (call, w, r, to - place[r])
                    if not torch.cuda.is_available():        # side by side they pass the checks, and then find no device
                        for to in (place[r] - sizes[w], place[r] + sizes[r] + (-sizes[r]) % 16):
                            assert calls(dict(place, **{w: to // 16 * 16}))[call]() == -5, (call, w, r)


def test_the_binding_refuses_what_the_library_cannot_see():
    pages, table = torch.zeros(2, 16, 576, dtype=torch.float16), torch.zeros(1, 2, dtype=torch.int32)
    with pytest.raises(ValueError, match="CUDA"):
        mla.mla_paged_gather(pages, table, None, torch.zeros(2, dtype=torch.int32), torch.zeros(1, 576).half())
    with pytest.raises(TypeError, match="float16 or torch.uint8"):
        binding._paged(pages.float(), table, -1)
    with pytest.raises(ValueError, match="576"):
        binding._paged(pages[..., :500], table, -1)
    with pytest.raises(ValueError, match="656"):
        binding._paged(pages.view(torch.uint8), table, -1)
    with pytest.raises(TypeError, match="int32"):
        binding._paged(pages, table.long(), -1)
    with pytest.raises(ValueError, match="max_pages"):
        binding._paged(pages, table[0], -1)
    with pytest.raises(ValueError, match="contiguous"):
        binding._paged(pages, torch.zeros(4, 3, dtype=torch.int32).t(), -1)


class OnDevice1(torch.Tensor):
    """A host tensor that says that it lies on CUDA device 1."""
    is_cuda, device = True, torch.device("cuda", 1)

    def get_device(self):
        return 1


class OnDevice0(OnDevice1):
    device = torch.device("cuda", 0)

    def get_device(self):
        return 0


def test_a_step_on_another_device_runs_all_its_calls_there(monkeypatch):
    """A stand-in for the library notes the current device and the stream of each call."""
    current, calls = [0], []

    class Device:
        def __init__(self, index):
            self.index = index

        def __enter__(self):
            self.before, current[0] = current[0], self.index

        def __exit__(self, *exc):
            current[0] = self.before

    class Lib:
        def __getattr__(self, name):
            def call(*args):
                stream = args[-1].value if isinstance(args[-1], ctypes.c_void_p) else args[-1]
                calls.append((name, current[0], stream))
                return 0
            return call

    class Stream:
        def __init__(self, handle):
            self.cuda_stream = handle

    monkeypatch.setattr(torch.cuda, "current_device", lambda: current[0])
    monkeypatch.setattr(torch.cuda, "device", Device)
    monkeypatch.setattr(torch.cuda, "current_stream", lambda *a: Stream(100 + current[0]))
    monkeypatch.setattr(binding, "_raw_stream", lambda dev: 100 + dev)
    monkeypatch.setattr(binding, "load_library", Lib)

    def on1(*shape, dtype=torch.bfloat16):
        return torch.zeros(*shape, dtype=dtype).as_subclass(OnDevice1)

    H, i32 = 16, torch.int32
    bufs = pipeline.PagedBuffers(on1(2, H, 512, dtype=torch.float16), on1(2, H, 512, dtype=torch.float16),
                                 on1(2, H, 128, dtype=torch.float32), on1(64, dtype=torch.uint8))
    args = dict(q_nope=on1(2, H, 128), q_pe=on1(2, H, 64), c_kv=on1(2, 512), k_pe=on1(2, 64), wk_b=on1(H, 128, 512),
                wv_b=on1(H, 512, 128), pages=on1(3, 16, 576, dtype=torch.float16), block_table=on1(1, 2, dtype=i32),
                cu_q=on1(2, dtype=i32), seq_len=on1(1, dtype=i32))
    pipeline.mla_paged_step(**args, bufs=bufs)
    assert [c[0] for c in calls] == ["mla_paged_append", "mla_absorb_q", "mla_attn_paged", "mla_late_decompress"]
    assert all(c[1:] == (1, 101) for c in calls), calls
    assert current[0] == 0
    # and none of them runs when the tensors lie on two devices
    del calls[:]
    for name in ("c_kv", "wk_b", "wv_b"):
        with pytest.raises(ValueError, match=name):
            pipeline.mla_paged_step(**dict(args, **{name: args[name].as_subclass(OnDevice0)}), bufs=bufs)
    bufs.o = bufs.o.as_subclass(OnDevice0)
    with pytest.raises(ValueError, match="bufs.o"):
        pipeline.mla_paged_step(**args, bufs=bufs)
    assert not calls


@pytest.mark.parametrize("kw", [dict(window=1 << 31), dict(window=(1 << 32) + 5), dict(n_sink=1 << 40),
                                dict(window=5 - (1 << 32))], ids=str)
def test_windows_past_32_bits_are_refused(monkeypatch, kw):
    monkeypatch.setattr(torch.cuda, "current_device", lambda: 1)

    class Lib:
        mla_attn_paged = None

    monkeypatch.setattr(binding, "load_library", Lib)

    def on1(*shape, dtype=torch.int32):
        return torch.zeros(*shape, dtype=dtype).as_subclass(OnDevice1)

    f16 = torch.float16
    with pytest.raises(ValueError, match="window"):
        mla.mla_attn_paged(on1(2, 16, 512, dtype=f16), on1(2, 16, 64, dtype=torch.bfloat16),
                           on1(3, 16, 576, dtype=f16), on1(1, 2), on1(2), on1(1), on1(2, 16, 512, dtype=f16),
                           workspace=on1(64, dtype=torch.uint8), **kw)


def test_a_workspace_that_is_no_tensor_is_refused_by_name(monkeypatch):
    monkeypatch.setattr(torch.cuda, "current_device", lambda: 1)

    class Lib:
        mla_attn_paged = None

    monkeypatch.setattr(binding, "load_library", Lib)

    def on1(*shape, dtype=torch.int32):
        return torch.zeros(*shape, dtype=dtype).as_subclass(OnDevice1)

    f16 = torch.float16
    for bad, error in ((1 << 20, TypeError), (bytearray(64), TypeError), (on1(64), TypeError),
                       (torch.zeros(64, dtype=torch.uint8), ValueError)):
        with pytest.raises(error, match="workspace"):
            mla.mla_attn_paged(on1(2, 16, 512, dtype=f16), on1(2, 16, 64, dtype=torch.bfloat16),
                               on1(3, 16, 576, dtype=f16), on1(1, 2), on1(2), on1(1), on1(2, 16, 512, dtype=f16),
                               workspace=bad)


def test_allocations_belong_to_the_stream_that_a_handle_names(monkeypatch):
    """Handles 0 and 1 are the default stream's; others are wrapped; Stream objects and None pass."""
    monkeypatch.setattr(torch.cuda, "stream", lambda s: s)
    monkeypatch.setattr(torch.cuda, "default_stream", lambda dev: ("default", dev))
    monkeypatch.setattr(torch.cuda, "ExternalStream", lambda h, device: ("external", h, device))

    class Foreign:
        def __init__(self, handle):
            self.cuda_stream = handle

    for h in (0, 1):
        assert binding.stream_context(h, 1) == binding.stream_context(Foreign(h), 1) == ("default", 1)
    assert binding.stream_context(0x7f00, 0) == binding.stream_context(Foreign(0x7f00), 0) == ("external", 0x7f00, 0)
    assert binding.stream_context(None, 0) is None


def test_oracle_rows():
    v = PO.e4m3_values()
    assert v[0x7E] == 448 and v[1] == 2.0 ** -9 and v[8] == 2.0 ** -6 and v[0x38] == 1.0 and v[0xB8] == -1.0
    t = torch.arange(256, dtype=torch.uint8).view(torch.float8_e4m3fn).double().numpy()
    assert np.array_equal(np.nan_to_num(v, nan=9), np.nan_to_num(t, nan=9))
    x = np.random.default_rng(0).uniform(-448, 448, 4000) * 2.0 ** -np.random.default_rng(1).integers(0, 17, 4000)
    x = np.concatenate([x, v[:0x7F], (v[:0x7E] + v[1:0x7F]) / 2])       # values, and ties between them
    assert np.array_equal(PO.e4m3_round(x), torch.from_numpy(x).float().to(torch.float8_e4m3fn).view(torch.uint8).numpy())
    lat = np.random.default_rng(2).standard_normal((5, 512)) * np.exp(np.linspace(-14, 9, 5))[:, None]
    raw = PO.pack_rows(lat, np.ones((5, 64)), True)
    assert raw.shape == (5, 656)
    back = PO.row_values(raw, True)
    big = np.abs(lat.reshape(5, 16, 32)).max(-1).repeat(32, axis=1).reshape(5, 512)
    # half a step of three mantissa bits, or of the smallest step under the block's scale
    assert (np.abs(back[:, :512] - lat) <= np.maximum(2.0 ** -4 * np.abs(lat), 2.0 ** -25 + 2.0 ** -17 * big)).all()
    assert (back[:, 512:] == 1).all()


def test_oracle_attention_is_the_masked_softmax():
    b = Batch(0, False, 16, 16, [3], [40], 9, 2)
    o, _ = b.ref()
    q = np.concatenate([b.q_lat, b.q_pe], -1).astype(np.float64)
    for i in range(3):
        p = 37 + i
        j = np.arange(40)
        s = (q[i] @ b.rows[0].T) * float(np.float32(1 / np.sqrt(192)))
        s[:, (j > p) | ((j <= p - 9) & (j >= 2))] = -np.inf
        w = np.exp(s - s.max(1, keepdims=True))
        assert np.allclose(o[i], (w / w.sum(1, keepdims=True)) @ b.rows[0][:, :512], rtol=1e-12, atol=1e-12)
