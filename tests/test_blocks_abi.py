"""Refusals of the normed append and of the calls with blocks, on the host (no GPU needed), and their oracle."""
import ctypes
import types

import numpy as np
import pytest
import torch

import mla_latent_kv_lat_gb300 as mla
from mla_latent_kv_lat_gb300 import binding, build, pipeline
from oracle import blocks_oracle as BO
from tests.test_paged_abi import BAD_CACHES, GOOD, ODD, ODD4, OnDevice0, OnDevice1, cache

FAR = 0x400000000                        # spans of their own, 16 GB apart; never dereferenced
NO_DEVICE = -5                           # what passes every check finds no device


def at(i):
    return FAR * (i + 1)


@pytest.fixture(scope="module")
def lib():
    build.build()
    return mla.load_library()


def dims(H=16, **kw):
    d = binding.make_dims(H)
    for k, v in kw.items():
        setattr(d, k, v)
    return ctypes.byref(d)


def calls(lib, B=2, T=4, H=16, K=3, n_scores=9, **kw):
    """name -> (arguments, call): every pointer a place of its own; ``kw`` replaces arguments by name."""
    ws = lib.mla_paged_workspace_size(dims())
    c = kw.pop("cache", None) or cache(pages=at(0), block_table=at(1), table_stride=9)
    base = dict(
        norm=dict(dims=dims(H), q=at(2), qt=H * 192, qh=192, kv=at(3), kt=576, qw=at(4), kw=at(5), cache=c, cu=at(6), len=at(7),
                  B=B, T=T, eps=1e-6, base=1e4, scale=1.0, q_nope=at(8), q_pe=at(9), stream=None),
        keys=dict(cache=c, cu=at(6), len=at(7), B=B, T=T, keys=at(8), stream=None),
        scores=dict(dims=dims(H), q_lat=at(2), q_pe=at(3), cache=c, keys=at(4), cu=at(6), len=at(7), B=B, T=T, scores=at(8),
                    ss=n_scores, n_scores=n_scores, stream=None),
        select=dict(scores=at(2), ss=n_scores, n_scores=n_scores, cu=at(6), len=at(7), B=B, T=T, n_sink=1, n_local=1,
                    blocks=at(8), counts=at(9), K=K, stream=None),
        attn=dict(dims=dims(H), q_lat=at(2), q_pe=at(3), cache=c, cu=at(6), len=at(7), B=B, T=T, blocks=at(4), counts=at(5), K=K,
                  ws=at(8), ws_bytes=ws, o=at(9), stream=None))
    fn = dict(norm=lib.mla_paged_norm_append, keys=lib.mla_paged_block_keys, scores=lib.mla_paged_block_scores,
              select=lib.mla_paged_select_blocks, attn=lib.mla_attn_paged_blocks)
    return {k: (v, lambda k=k, **new: fn[k](*{**base[k], **new}.values())) for k, v in base.items()}


def test_good_arguments_pass_the_checks(lib):
    if torch.cuda.is_available():
        pytest.skip("addresses of nobody must not reach a device")
    for name, (_, call) in calls(lib).items():
        assert call() == NO_DEVICE, name
    c = calls(lib)
    assert c["norm"][1](qw=None) == NO_DEVICE and c["norm"][1](qt=0, qh=0, kt=0) == NO_DEVICE
    assert c["select"][1](K=1024, n_sink=1000, n_local=24) == NO_DEVICE
    assert c["attn"][1](K=1024) == NO_DEVICE
    assert calls(lib, T=1)["select"][1](ss=0) == NO_DEVICE
    assert calls(lib, T=1)["scores"][1](ss=0) == NO_DEVICE


def test_lists_need_no_workspace_of_their_own(lib):
    """Partials and records of each pair of SMs, and the staging with its table: what attention over whole contexts
    needs.  A buffer of that size serves both calls."""
    partials = lib.mla_paged_workspace_size(dims()) - (131072 * 1024 + 4096)
    assert partials > 0 and partials % (2 * 128 * (512 + 2) * 4 + 32) == 0


def test_bad_caches_are_refused(lib):
    for kw, want in BAD_CACHES + [(dict(page_size=32), -2), (dict(page_size=16), -2)]:
        for name, (_, call) in calls(lib).items():
            if name == "select" or (name == "norm" and kw.get("page_size") in (16, 32)):
                continue                 # has no cache; takes any page
            if name == "scores" and not {"pages", "type"}.isdisjoint(kw):
                continue                 # looks at neither
            bad = cache(**dict(dict(pages=at(0), block_table=at(1), table_stride=9), **kw))
            assert call(cache=bad) == want, (name, kw)
    for name in ("norm", "keys", "scores", "attn"):
        assert calls(lib)[name][1](cache=None) == -1, name


BAD = [
    ("norm", dict(q=None), -1), ("norm", dict(kv=None), -1), ("norm", dict(kw=None), -1), ("norm", dict(q_nope=None), -1),
    ("norm", dict(q_pe=None), -1), ("norm", dict(cu=None), -1), ("norm", dict(len=None), -1), ("norm", dict(B=0), -1),
    ("norm", dict(T=0), -1), ("norm", dict(T=-1), -1), ("norm", dict(qt=-8), -1), ("norm", dict(qh=-8), -1),
    ("norm", dict(kt=-8), -1), ("norm", dict(qt=16 * 192 + 4), -3), ("norm", dict(qh=194), -3), ("norm", dict(kt=577), -3),
    ("norm", dict(q=ODD), -3), ("norm", dict(kv=ODD), -3), ("norm", dict(qw=ODD), -3), ("norm", dict(kw=ODD), -3),
    ("norm", dict(q_nope=ODD), -3), ("norm", dict(q_pe=ODD), -3), ("norm", dict(cu=ODD4), -3), ("norm", dict(len=ODD4), -3),
    ("norm", dict(eps=0.0), -1), ("norm", dict(eps=-1.0), -1), ("norm", dict(eps=float("nan")), -1),
    ("norm", dict(eps=float("inf")), -1), ("norm", dict(base=1.0), -1), ("norm", dict(scale=0.0), -1),
    ("norm", dict(scale=float("nan")), -1), ("norm", dict(T=1 << 28), -2), ("norm", dict(qt=1 << 40), -2),
    ("norm", dict(kt=1 << 62), -2), ("norm", dict(qh=1 << 50), -2),
    ("keys", dict(keys=None), -1), ("keys", dict(keys=ODD), -3), ("keys", dict(cu=None), -1), ("keys", dict(len=ODD4), -3),
    ("keys", dict(T=0), -1), ("keys", dict(B=0), -1),
    ("scores", dict(q_lat=None), -1), ("scores", dict(q_pe=ODD), -3), ("scores", dict(keys=None), -1), ("scores", dict(keys=ODD), -3),
    ("scores", dict(scores=None), -1), ("scores", dict(scores=ODD4), -3), ("scores", dict(T=0), -1), ("scores", dict(B=0), -1),
    ("scores", dict(n_scores=0), -1), ("scores", dict(ss=8), -1), ("scores", dict(ss=-9), -1), ("scores", dict(T=1 << 28), -2),
    ("scores", dict(ss=1 << 40), -2), ("scores", dict(cu=ODD4), -3),
    ("select", dict(scores=None), -1), ("select", dict(blocks=None), -1), ("select", dict(counts=None), -1),
    ("select", dict(scores=ODD4), -3), ("select", dict(blocks=ODD4), -3), ("select", dict(counts=ODD4), -3),
    ("select", dict(T=0), -1), ("select", dict(B=0), -1), ("select", dict(n_scores=0), -1), ("select", dict(ss=8), -1),
    ("select", dict(n_sink=-1), -1), ("select", dict(n_local=0), -1), ("select", dict(K=0), -1), ("select", dict(n_sink=2, n_local=2), -1),
    ("select", dict(n_sink=2 ** 31 - 1, n_local=2 ** 31 - 1), -1), ("select", dict(K=1025), -2), ("select", dict(B=65536), -2),
    ("select", dict(ss=1 << 40), -2), ("select", dict(ss=1 << 26, n_scores=1 << 26), -2),
    ("scores", dict(ss=1 << 26, n_scores=1 << 26), -2), ("scores", dict(ss=2 ** 31 - 1, n_scores=2 ** 31 - 1), -2),
    ("attn", dict(blocks=None), -1), ("attn", dict(counts=None), -1), ("attn", dict(blocks=ODD4), -3), ("attn", dict(counts=ODD4), -3),
    ("attn", dict(K=0), -1), ("attn", dict(K=-1), -1), ("attn", dict(K=1025), -2), ("attn", dict(T=0), -1), ("attn", dict(B=0), -1),
    ("attn", dict(q_lat=None), -1), ("attn", dict(o=ODD), -3), ("attn", dict(ws=None), -4), ("attn", dict(ws_bytes=16), -4),
    ("attn", dict(ws=ODD), -3), ("attn", dict(T=1 << 28), -2), ("attn", dict(cu=None), -1)]


@pytest.mark.parametrize("name,kw,want", BAD, ids=[f"{n}-{k}" for n, k, _ in BAD])
def test_bad_arguments_are_refused(lib, name, kw, want):
    assert calls(lib)[name][1](**kw) == want


def test_bad_dims_are_refused(lib):
    for name in ("norm", "scores", "attn"):
        call = calls(lib)[name][1]
        assert call(dims=None) == -1 and call(dims=dims(24)) == -2 and call(dims=dims(144)) == -2, name
        assert call(dims=dims(16, qk_rope=32)) == -2 and call(dims=dims(16, scale=0.0)) == -1, name


def test_overlapping_memory_is_refused(lib):
    """What a call writes, laid over the first and the last 16 (or 4) bytes of each thing that it reads or writes."""
    B, T, H, K, W = 3, 5, 16, 7, 11
    for type_, row in ((0, 1152), (1, 656)):
        ws = lib.mla_paged_workspace_size(dims())
        common = dict(pages=100 * 64 * row, table=((B - 1) * 9 + 8) * 4, cu=4 * (B + 1), len=4 * B)
        sizes = dict(
            norm=dict(common, q=2 * (4 * (H * 192 + 8) + H * 192), kv=2 * (4 * 584 + 576), qw=384, kw=1024, q_nope=T * H * 256,
                      q_pe=T * H * 128),
            keys=dict(common, keys=100 * 1152),
            scores=dict(table=common["table"], cu=common["cu"], len=common["len"], q_lat=T * H * 1024, q_pe=T * H * 128,
                        keys=100 * 1152, scores=4 * (4 * (W + 2) + W)),
            select=dict(cu=common["cu"], len=common["len"], scores=4 * (4 * (W + 2) + W), blocks=4 * T * K, counts=4 * T),
            attn=dict(common, q_lat=T * H * 1024, q_pe=T * H * 128, blocks=4 * T * K, counts=4 * T, ws=ws, o=T * H * 1024))
        writes = dict(norm=("q_nope", "q_pe", "pages"), keys=("keys",), scores=("scores",), select=("blocks", "counts"),
                      attn=("o", "ws"))
        for name, size in sizes.items():
            place = {k: at(i) for i, k in enumerate(size)}

            def go(place):
                c = cache(pages=place.get("pages", at(30)), block_table=place.get("table", at(31)), table_stride=9, type=type_)
                new = {k: v for k, v in place.items() if k not in ("pages", "table")}
                if name == "norm":
                    new.update(qt=H * 192 + 8, kt=584)
                if name in ("scores", "select"):
                    new.update(ss=W + 2, n_scores=W)
                if name in ("select", "attn"):
                    new["K"] = K
                if name != "select":
                    new["cache"] = c
                return calls(lib)[name][1](B=B, T=T, **new)

            if not torch.cuda.is_available():
                assert go(place) == NO_DEVICE, name
            for w in writes[name]:
                step = 4 if w in ("blocks", "counts", "scores") else 16
                for r in size:
                    if r == w:
                        continue
                    first, last = place[r] - size[w] + step, place[r] + (size[r] - 1) // step * step
                    for to in (first + (-first) % step, last):
                        assert go(dict(place, **{w: to})) == -1, (name, w, r, to - place[r])
                    if not torch.cuda.is_available():    # side by side they pass the checks
                        for to in (place[r] - size[w], place[r] + size[r] + (-size[r]) % 16):
                            assert go(dict(place, **{w: to // 16 * 16})) == NO_DEVICE, (name, w, r)


# ---------------------------------------------------------------------------
# the binding
# ---------------------------------------------------------------------------
def on1(*shape, dtype=torch.int32):
    return torch.zeros(*shape, dtype=dtype).as_subclass(OnDevice1)


BF, F16, F32, U8 = torch.bfloat16, torch.float16, torch.float32, torch.uint8


def good():
    H = 16
    return dict(
        norm=(mla.mla_paged_norm_append, dict(q=on1(2, H, 192, dtype=BF), kv=on1(2, 576, dtype=BF), q_weight=on1(192, dtype=BF),
                                             kv_weight=on1(512, dtype=BF), pages=on1(3, 64, 576, dtype=F16),
                                             block_table=on1(1, 2), cu_new=on1(2), seq_len=on1(1),
                                             q_nope=on1(2, H, 128, dtype=BF), q_pe=on1(2, H, 64, dtype=BF))),
        keys=(mla.mla_paged_block_keys, dict(pages=on1(3, 64, 576, dtype=F16), block_table=on1(1, 2), cu_new=on1(2),
                                             seq_len=on1(1), block_keys=on1(3, 1, 576, dtype=F16), T=2)),
        scores=(mla.mla_paged_block_scores, dict(q_lat=on1(2, H, 512, dtype=F16), q_pe=on1(2, H, 64, dtype=BF),
                                                 block_keys=on1(3, 1, 576, dtype=F16), block_table=on1(1, 2), cu_q=on1(2),
                                                 seq_len=on1(1), scores=on1(2, 5, dtype=F32))),
        select=(mla.mla_paged_select_blocks, dict(scores=on1(2, 5, dtype=F32), cu_q=on1(2), seq_len=on1(1), blocks=on1(2, 3),
                                                  counts=on1(2))),
        attn=(mla.mla_attn_paged_blocks, dict(q_lat=on1(2, H, 512, dtype=F16), q_pe=on1(2, H, 64, dtype=BF),
                                              pages=on1(3, 64, 576, dtype=F16), block_table=on1(1, 2), cu_q=on1(2), seq_len=on1(1),
                                              blocks=on1(2, 3), counts=on1(2), o_lat=on1(2, H, 512, dtype=F16),
                                              workspace=on1(64, dtype=U8))))


@pytest.fixture
def device1(monkeypatch, lib):
    """Device 1 is current; a stand-in for the library notes its calls."""
    seen = []

    class Lib:
        def __getattr__(self, name):
            return lambda *args: seen.append(name) or 0

    monkeypatch.setattr(torch.cuda, "current_device", lambda: 1)
    monkeypatch.setattr(binding, "_raw_stream", lambda dev: 100 + dev)
    binding._fast()                      # (with the library that there is)
    monkeypatch.setattr(binding, "load_library", Lib)
    return seen


def test_the_binding_takes_good_tensors(device1):
    for name, (fn, kw) in good().items():
        fn(**kw)
        assert device1.pop() == fn.__name__, name
    fn, kw = good()["norm"]
    fn(**dict(kw, q_weight=None))
    fn(**dict(kw, q=on1(2, 16 * 192 + 64, dtype=BF)[:, 64:].unflatten(1, (16, 192)).as_subclass(OnDevice1)))
    fn, kw = good()["select"]
    fn(**dict(kw, scores=on1(2, 9, dtype=F32)[:, :5].as_subclass(OnDevice1)))


SHAPES = [("norm", "q", on1(2, 16, 191, dtype=BF)), ("norm", "q", on1(2, 16 * 192, dtype=BF)), ("norm", "kv", on1(3, 576, dtype=BF)),
          ("norm", "kv", on1(2, 577, dtype=BF)), ("norm", "q_weight", on1(128, dtype=BF)), ("norm", "kv_weight", on1(576, dtype=BF)),
          ("norm", "q_nope", on1(2, 16, 64, dtype=BF)), ("norm", "q_pe", on1(2, 64, dtype=BF)), ("norm", "cu_new", on1(3)),
          ("norm", "seq_len", on1(2)), ("keys", "block_keys", on1(3, 2, 576, dtype=F16)), ("keys", "block_keys", on1(2, 1, 576, dtype=F16)),
          ("scores", "scores", on1(3, 5, dtype=F32)), ("scores", "scores", on1(10, dtype=F32)), ("scores", "scores", on1(2, 0, dtype=F32)),
          ("scores", "block_keys", on1(3, 1, 512, dtype=F16)), ("scores", "block_keys", on1(3, 576, dtype=F16)),
          ("scores", "q_pe", on1(2, 8, 64, dtype=BF)), ("select", "blocks", on1(6)), ("select", "counts", on1(3)),
          ("select", "scores", on1(1, 5, dtype=F32)), ("attn", "blocks", on1(3, 3)), ("attn", "blocks", on1(6)),
          ("attn", "counts", on1(2, 1)), ("attn", "o_lat", on1(2, 16, 511, dtype=F16))]


@pytest.mark.parametrize("name,arg,bad", SHAPES, ids=[f"{n}-{a}-{tuple(t.shape)}" for n, a, t in SHAPES])
def test_the_binding_refuses_wrong_shapes_by_name(device1, name, arg, bad):
    fn, kw = good()[name]
    with pytest.raises(ValueError, match=arg):
        fn(**dict(kw, **{arg: bad}))
    assert not device1


TYPES = [("norm", "q", F16), ("norm", "kv", F32), ("norm", "kv_weight", F32), ("norm", "q_pe", F16), ("keys", "block_keys", BF),
         ("scores", "block_keys", BF), ("scores", "scores", F16), ("scores", "q_lat", BF), ("select", "blocks", torch.int64),
         ("select", "scores", torch.float64), ("attn", "blocks", torch.int64), ("attn", "counts", torch.int64), ("attn", "workspace", torch.int8)]


@pytest.mark.parametrize("name,arg,dtype", TYPES, ids=[f"{n}-{a}" for n, a, _ in TYPES])
def test_the_binding_refuses_wrong_types_by_name(device1, name, arg, dtype):
    fn, kw = good()[name]
    with pytest.raises(TypeError, match=arg):
        fn(**dict(kw, **{arg: kw[arg].to(dtype).as_subclass(OnDevice1)}))
    assert not device1


def test_the_binding_refuses_other_devices_and_layouts(device1):
    for name, (fn, kw) in good().items():
        for arg, t in kw.items():
            if not isinstance(t, torch.Tensor) or arg == next(iter(kw)):
                continue
            with pytest.raises(ValueError):
                fn(**dict(kw, **{arg: t.as_subclass(OnDevice0)}))
    for name, arg in (("norm", "q_nope"), ("scores", "q_lat"), ("attn", "blocks"), ("select", "blocks"), ("keys", "block_keys")):
        fn, kw = good()[name]
        t = kw[arg]
        with pytest.raises(ValueError, match="contiguous"):
            fn(**dict(kw, **{arg: torch.cat([t, t], -1)[..., ::2].as_subclass(OnDevice1)}))
    for name, arg in (("norm", "q"), ("norm", "kv"), ("scores", "scores"), ("select", "scores")):
        fn, kw = good()[name]
        t = kw[arg]
        with pytest.raises(ValueError, match="last dimension"):
            fn(**dict(kw, **{arg: torch.cat([t, t], -1)[..., ::2].as_subclass(OnDevice1)}))
    fn, kw = good()["select"]
    for bad in (dict(n_sink=1 << 31), dict(n_local=-1 << 40)):
        with pytest.raises(ValueError, match="int32"):
            fn(**kw, **bad)
    fn, kw = good()["keys"]
    with pytest.raises(ValueError, match="int32"):
        fn(**dict(kw, T=1 << 32))
    assert not device1


def test_the_compiled_way_leaves_what_is_not_plainly_right_to_the_binding(lib):
    """It returns None for tensors that are on no GPU, for no tensors, and for too few arguments."""
    fast = binding._fast()
    cpu = torch.zeros(2, 16, 512, dtype=F16)
    for f, n in ((fast.append, 9), (fast.gather, 6), (fast.attn, 12), (fast.norm_append, 14), (fast.block_keys, 7), (fast.block_scores, 9), (fast.select_blocks, 8), (fast.attn_blocks, 12)):
        assert f(*[cpu] * n) is None and f(*[None] * n) is None and f(*[3.5] * n) is None and f() is None
        assert f(*[cpu] * (n + 1)) is None


def test_without_the_compiled_module_the_calls_go_through_python(monkeypatch, device1, tmp_path):
    monkeypatch.setattr(binding, "_calls", None)
    monkeypatch.setattr(build, "calls_path", lambda: str(tmp_path / "_calls_of_another.so"))
    with pytest.warns(UserWarning, match="_calls_of_another"):
        binding._fast()
    for name, (fn, kw) in good().items():
        fn(**kw)
        assert device1.pop() == fn.__name__, name


def test_the_library_is_built_without_the_module_where_that_cannot_be(monkeypatch, tmp_path):
    def calls():
        raise AssertionError("no compiler")

    made = []
    monkeypatch.setattr(build, "LIB", str(tmp_path / "libmla.so"))
    monkeypatch.setattr(build, "BUILD", str(tmp_path))
    monkeypatch.setattr(build, "calls_path", lambda: str(tmp_path / "_calls.so"))
    monkeypatch.setattr(build, "_build_calls", calls)
    monkeypatch.setattr(build, "_compile", lambda src, extra: made.append(src) or src)
    def link(cmd, **kw):
        open(build.LIB + ".tmp", "w").close()
        return types.SimpleNamespace(returncode=0)

    monkeypatch.setattr(build.subprocess, "run", link)
    monkeypatch.setattr(build, "can_build_calls", lambda: False)
    assert not build.up_to_date()
    assert build.build() == build.LIB and made and build.up_to_date()
    monkeypatch.setattr(build, "can_build_calls", lambda: True)
    assert not build.up_to_date()
    with pytest.raises(AssertionError, match="no compiler"):
        build.build()


def test_a_step_on_another_device_runs_all_its_calls_there(monkeypatch, lib):
    """A stand-in for the library notes the current device and the stream of each call."""
    current, seen = [0], []

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
                seen.append((name, current[0], stream))
                return 0
            return call

    class Stream:
        def __init__(self, handle):
            self.cuda_stream = handle

    binding._fast()
    monkeypatch.setattr(torch.cuda, "current_device", lambda: current[0])
    monkeypatch.setattr(torch.cuda, "device", Device)
    monkeypatch.setattr(torch.cuda, "current_stream", lambda *a: Stream(100 + current[0]))
    monkeypatch.setattr(binding, "_raw_stream", lambda dev: 100 + dev)
    monkeypatch.setattr(binding, "load_library", Lib)
    H = 16
    bufs = pipeline.SparseBuffers(on1(2, H, 128, dtype=BF), on1(2, H, 64, dtype=BF), on1(2, H, 512, dtype=F16), on1(2, 2, dtype=F32),
                                  on1(2, 3), on1(2), on1(2, H, 512, dtype=F16), on1(2, H, 128, dtype=F32), on1(64, dtype=U8))
    args = dict(q=on1(2, H, 192, dtype=BF), kv=on1(2, 576, dtype=BF), q_weight=None, kv_weight=on1(512, dtype=BF),
                wk_b=on1(H, 128, 512, dtype=BF), wv_b=on1(H, 512, 128, dtype=BF), pages=on1(3, 64, 576, dtype=F16),
                block_keys=on1(3, 1, 576, dtype=F16), block_table=on1(1, 2), cu_q=on1(2), seq_len=on1(1))
    args["n_blocks"] = 3
    pipeline.mla_paged_sparse_step(**args, bufs=bufs)
    assert [c[0] for c in seen] == ["mla_paged_norm_append", "mla_paged_block_keys", "mla_absorb_q", "mla_paged_block_scores",
                                    "mla_paged_select_blocks", "mla_attn_paged_blocks", "mla_late_decompress"]
    assert all(c[1:] == (1, 101) for c in seen), seen
    assert current[0] == 0
    del seen[:]
    for name in ("wk_b", "wv_b"):
        with pytest.raises(ValueError, match=name):
            pipeline.mla_paged_sparse_step(**dict(args, **{name: args[name].as_subclass(OnDevice0)}), bufs=bufs)
    bufs.o = bufs.o.as_subclass(OnDevice0)
    with pytest.raises(ValueError, match="bufs.o"):
        pipeline.mla_paged_sparse_step(**args, bufs=bufs)
    with pytest.raises(ValueError, match="n_blocks"):
        pipeline.mla_paged_sparse_step(**dict(args, n_blocks=4), bufs=bufs)
    assert not seen


# ---------------------------------------------------------------------------
# the oracle
# ---------------------------------------------------------------------------
def test_oracle_by_loops():
    rng = np.random.default_rng(0)
    x, w = rng.standard_normal((3, 5)), rng.standard_normal(5)
    for i in range(3):
        r = (sum(v * v for v in x[i]) / 5 + 0.25) ** 0.5
        assert np.allclose(BO.rms(x, w, 0.25)[i], [v / r * u for v, u in zip(x[i], w)])
    assert np.array_equal(BO.rms(x, None, 0.25), x)
    rows = rng.standard_normal((150, 576))
    m = BO.mean_rows(rows)
    assert m.shape == (2, 576) and np.allclose(m[1], sum(rows[64 + i] for i in range(64)) / 64)
    q = rng.standard_normal((2, 3, 576))
    s, mag = BO.block_scores(q, m, 127, 4, 0.5)                  # positions 127 (own block 1) and 128 (own block 2)
    assert np.isneginf(s[0, 1:]).all() and np.isneginf(s[1, 2:]).all()
    assert np.allclose(s[1, 1], 0.5 * max(sum(q[1, h, c] * m[1, c] for c in range(576)) for h in range(3)))
    assert (mag[1, :2] >= np.abs(s[1, :2])).all()
    sc = np.array([1.0, 5.0, np.nan, 5.0, -np.inf, 7.0, 2.0, 3.0])
    assert list(BO.select(sc, 64 * 7 + 1, 4, 1, 2)) == [0, 5, 6, 7]       # own 7, before it 6, first 0, and the best
    assert list(BO.select(sc, 64 * 7 + 1, 4, 0, 1)) == [1, 3, 5, 7]
    assert list(BO.select(sc, 64 * 7 + 1, 3, 0, 1)) == [1, 5, 7]          # of 1 and 3, the same, the lower
    assert list(BO.select(sc, 64 * 7 + 1, 8, 0, 1)) == list(range(8))
    assert list(BO.select(sc, 64 * 5, 5, 0, 1)) == [0, 1, 3, 4, 5]       # NaN ranks below -inf
    assert list(BO.select(sc, 10, 4, 2, 2)) == [0]
    o, a, n = BO.attend_blocks(q[0], rows, 140, [2, 0, 0], 0.1)
    keys = list(range(128, 141)) + list(range(64)) * 2
    e = np.exp(0.1 * q[0] @ rows[keys].T)
    assert n == len(keys) and np.allclose(o, (e / e.sum(1, keepdims=True)) @ rows[keys][:, :512]) and (a >= np.abs(o)).all()
    o, a, n = BO.attend_blocks(q[0], rows, 140, [], 0.1)
    assert n == 0 and not o.any()
