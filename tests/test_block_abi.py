"""Host-side checks of the block-scaled and block-sparse calls: every refusal
comes before a launch, so none of these needs a GPU."""
import ctypes
import types

import pytest
import torch

FAKE = 1 << 20  # a 256-byte aligned non-null value; never dereferenced here
P, I, I64, F, SZ = (ctypes.c_void_p, ctypes.c_int, ctypes.c_int64, ctypes.c_float, ctypes.c_size_t)
INVALID, UNSUPPORTED, WORKSPACE = 1, 2, 3


@pytest.fixture(scope="module")
def pa():
    from __graft_entry__ import build_library
    build_library()
    import paged_kv_cache_136_gb300 as pa
    return pa


def _caller(pa, name, spec):
    """fn(**changes) calling C entry `name` with spec's values, changed."""
    fn = getattr(ctypes.CDLL(pa.lib_path()), name)
    fn.restype = I
    fn.argtypes = [t for _, t, _ in spec]

    def call(**kw):
        values = {n: v for n, _, v in spec}
        assert set(kw) <= set(values)
        values.update(kw)
        return fn(*[values[n] for n, _, _ in spec])
    return call


REQ = [("tables", P, FAKE), ("table_stride", I64, 10), ("seq_lens", P, FAKE), ("qsl", P, FAKE),
       ("R", I, 4)]
SIZES = [("Hkv", I, 2), ("D", I, 128), ("bs", I, 16), ("NB", I, 100), ("MB", I, 10)]
WRITE = [("key", P, FAKE), ("value", P, FAKE), ("pool", P, FAKE), ("scales", P, FAKE), *REQ,
         ("T", I, 4), ("mq", I, 1), *SIZES, ("ks", I64, 256), ("vs", I64, 256), ("dtype", I, 0),
         ("stream", P, None)]
BOUNDS = [("bounds", P, FAKE), ("bsc", P, FAKE), ("pool", P, FAKE), ("scales", P, None), *REQ,
          ("mq", I, 1), *SIZES, ("dtype", I, 0), ("stream", P, None)]
SELECT = [("lists", P, FAKE), ("lens", P, FAKE), ("q", P, FAKE), ("bounds", P, FAKE),
          ("bsc", P, FAKE), ("tables", P, FAKE), ("seq_lens", P, FAKE), ("B", I, 4), ("H", I, 8),
          *SIZES, ("K", I, 5), ("sink", I, 1), ("recent", I, 1), ("dtype", I, 0), ("msl", I, 160),
          ("ws", P, FAKE), ("wb", SZ, 1 << 20), ("stream", P, None)]
DENSE = [("out", P, FAKE), ("lse", P, None), ("q", P, FAKE), ("pool", P, FAKE),
         ("scales", P, FAKE), ("tables", P, FAKE), ("seq_lens", P, FAKE), ("B", I, 4), ("H", I, 8),
         *SIZES, ("scale", F, 0.1), ("dtype", I, 0), ("msl", I, 160), ("ws", P, FAKE),
         ("wb", SZ, 1 << 30), ("stream", P, None)]
SPARSE = [("out", P, FAKE), ("lse", P, None), ("q", P, FAKE), ("pool", P, FAKE),
          ("scales", P, None), ("tables", P, FAKE), ("seq_lens", P, FAKE), ("lists", P, FAKE),
          ("lens", P, FAKE), ("B", I, 4), ("H", I, 8), *SIZES, ("K", I, 5), ("scale", F, 0.1),
          ("dtype", I, 0), ("ws", P, FAKE), ("wb", SZ, 1 << 30), ("stream", P, None)]

COMMON = [(dict(Hkv=0), INVALID), (dict(NB=0), INVALID), (dict(MB=0), INVALID),
          (dict(bs=0), INVALID), (dict(D=0), INVALID), (dict(seq_lens=0), INVALID),
          (dict(tables=0), INVALID), (dict(tables=FAKE + 2), INVALID), (dict(D=96), UNSUPPORTED),
          (dict(bs=8), UNSUPPORTED), (dict(dtype=4), UNSUPPORTED),
          (dict(NB=1 << 27), UNSUPPORTED)]
REQUESTS = COMMON + [(dict(R=-1), INVALID), (dict(mq=-1), INVALID), (dict(qsl=0), INVALID),
                     (dict(table_stride=9), INVALID), (dict(R=65536), UNSUPPORTED),
                     (dict(pool=0), INVALID), (dict(pool=FAKE + 8), INVALID)]
QUERIES = COMMON + [(dict(B=-1), INVALID), (dict(H=7), INVALID), (dict(q=0), INVALID),
                    (dict(q=FAKE + 8), INVALID), (dict(H=6), UNSUPPORTED),
                    (dict(H=32), UNSUPPORTED), (dict(B=65536), UNSUPPORTED), (dict(ws=0), WORKSPACE),
                    (dict(ws=FAKE + 128), WORKSPACE), (dict(wb=100), WORKSPACE)]
DECODE = QUERIES + [(dict(out=0), INVALID), (dict(out=FAKE + 4), INVALID),
                    (dict(lse=FAKE + 2), INVALID), (dict(scale=float("nan")), INVALID),
                    (dict(scale=float("inf")), INVALID), (dict(pool=0), INVALID)]


@pytest.mark.parametrize("kw,status", REQUESTS + [
    (dict(key=0), INVALID), (dict(value=FAKE + 8), INVALID), (dict(scales=0), INVALID),
    (dict(ks=255), INVALID), (dict(vs=260), INVALID), (dict(T=-1), INVALID)])
def test_write_refusals(pa, kw, status):
    assert _caller(pa, "pa_reshape_and_cache_fp8_block", WRITE)(**kw) == status


@pytest.mark.parametrize("kw,status", REQUESTS + [
    (dict(bounds=0), INVALID), (dict(bounds=FAKE + 8), INVALID), (dict(bsc=0), INVALID),
    (dict(scales=FAKE + 1), INVALID)])
def test_bounds_refusals(pa, kw, status):
    assert _caller(pa, "pa_update_block_bounds", BOUNDS)(**kw) == status


@pytest.mark.parametrize("kw,status", QUERIES + [
    (dict(K=0), INVALID), (dict(sink=-1), INVALID), (dict(sink=3, recent=3), INVALID),
    (dict(sink=2 ** 31 - 1, recent=2 ** 31 - 1), INVALID), (dict(msl=-1), INVALID),
    (dict(lists=0), INVALID), (dict(lens=0), INVALID), (dict(bounds=0), INVALID),
    (dict(bsc=0), INVALID)])
def test_select_refusals(pa, kw, status):
    assert _caller(pa, "pa_select_blocks", SELECT)(**kw) == status


@pytest.mark.parametrize("kw,status", DECODE + [(dict(scales=0), INVALID), (dict(msl=-1), INVALID)])
def test_decode_refusals(pa, kw, status):
    assert _caller(pa, "pa_decode_fp8_block", DENSE)(**kw) == status


@pytest.mark.parametrize("kw,status", DECODE + [
    (dict(K=0), INVALID), (dict(lists=0), INVALID), (dict(lens=0), INVALID),
    (dict(lists=FAKE + 1), INVALID)])
def test_sparse_refusals(pa, kw, status):
    assert _caller(pa, "pa_decode_sparse", SPARSE)(**kw) == status


def test_nothing_to_do_is_ok(pa):
    assert _caller(pa, "pa_reshape_and_cache_fp8_block", WRITE)(R=0) == 0
    assert _caller(pa, "pa_reshape_and_cache_fp8_block", WRITE)(T=0) == 0
    assert _caller(pa, "pa_reshape_and_cache_fp8_block", WRITE)(mq=0) == 0
    assert _caller(pa, "pa_update_block_bounds", BOUNDS)(R=0) == 0
    assert _caller(pa, "pa_update_block_bounds", BOUNDS)(mq=0) == 0
    assert _caller(pa, "pa_select_blocks", SELECT)(B=0) == 0
    assert _caller(pa, "pa_decode_fp8_block", DENSE)(B=0) == 0
    assert _caller(pa, "pa_decode_sparse", SPARSE)(B=0) == 0


def test_workspace_sizes(pa):
    assert pa.pa_block_decode_workspace_size(32, 8, 128) > 0
    assert pa.pa_block_decode_workspace_size(32, 7, 128) == 0
    assert pa.pa_block_decode_workspace_size(0, 8, 128) == 0
    # one 32-bit key for each (sequence, kv head, block), rounded up
    assert pa.pa_select_blocks_workspace_size(3, 2, 100, 16) >= 3 * 2 * 7 * 4
    assert pa.pa_select_blocks_workspace_size(0, 2, 100, 16) > 0
    assert pa.pa_select_blocks_workspace_size(3, 0, 100, 16) == 0


# ---------------------------------------------------------------------------
# The binding
# ---------------------------------------------------------------------------
def _args(nb=6, bs=16, hkv=2, d=64, b=3, h=4, mb=2, k=2):
    i32 = dict(dtype=torch.int32)
    return types.SimpleNamespace(
        key=torch.zeros(b, hkv, d, dtype=torch.float16), pool=torch.zeros(2, nb, bs, hkv, d,
                                                                         dtype=torch.uint8),
        pool16=torch.zeros(2, nb, bs, hkv, d, dtype=torch.float16), scales=torch.ones(2, nb, hkv),
        tables=torch.zeros(b, mb, **i32), sl=torch.ones(b, **i32), qsl=torch.arange(b + 1, **i32),
        q=torch.zeros(b, h, d, dtype=torch.float16), bounds=torch.zeros(nb, hkv, 2, d,
                                                                       dtype=torch.int8),
        bsc=torch.ones(nb, hkv), lists=torch.zeros(b, hkv, k, **i32), lens=torch.zeros(b, **i32),
        ws=torch.zeros(64, dtype=torch.uint8), bs=bs)


def _calls(pa, a):
    return {
        "write": lambda: pa.pa_reshape_and_cache_fp8_block(a.key, a.key, a.pool, a.scales, a.tables,
                                                           a.sl, a.qsl, a.bs, 1),
        "decode": lambda: pa.pa_decode_fp8_block(torch.empty_like(a.q), a.q, a.pool, a.scales,
                                                 a.tables, a.sl, 0.1, a.bs, 16, a.ws),
        "bounds": lambda: pa.pa_update_block_bounds(a.bounds, a.bsc, a.pool, a.tables, a.sl, a.qsl,
                                                    a.bs, 1, kv_scales=a.scales),
        "select": lambda: pa.pa_select_blocks(a.lists, a.lens, a.q, a.bounds, a.bsc, a.tables, a.sl,
                                              a.bs, 16, a.ws),
        "sparse": lambda: pa.pa_decode_sparse(torch.empty_like(a.q), a.q, a.pool16, a.tables, a.sl,
                                              a.lists, a.lens, 0.1, a.bs, a.ws),
    }


CALLS = ["write", "decode", "bounds", "select", "sparse"]


@pytest.mark.parametrize("name", CALLS)
def test_binding_wants_cuda_tensors(pa, name):
    with pytest.raises(ValueError, match="must be a CUDA tensor"):
        _calls(pa, _args())[name]()


class _Elsewhere:
    """A CPU tensor that says it lies on another device."""

    def __init__(self, tensor, device):
        self.tensor, self.device = tensor, device

    def get_device(self):
        return self.device

    def __getattr__(self, name):
        return getattr(self.tensor, name)


def test_binding_wants_the_current_device(pa):
    """Every tensor of a call on cuda:1 while cuda:0 is current, or one of them."""
    calls = pa._block_calls
    calls.bind(pa.PAError, lambda: 0, lambda device: 0)
    try:
        fields = [f for f in vars(_args()) if f != "bs"]
        a = _args()
        for f in fields:
            setattr(a, f, _Elsewhere(getattr(a, f), 1))
        for name, first in (("write", "key"), ("bounds", "bounds"), ("select", "block_lists")):
            with pytest.raises(ValueError, match=first + " must be on the current device, cuda:0"):
                _calls(pa, a)[name]()
        for call in (lambda out: pa.pa_decode_fp8_block(out, a.q, a.pool, a.scales, a.tables, a.sl,
                                                        0.1, a.bs, 16, a.ws),
                     lambda out: pa.pa_decode_sparse(out, a.q, a.pool16, a.tables, a.sl, a.lists,
                                                     a.lens, 0.1, a.bs, a.ws)):
            with pytest.raises(ValueError, match="out must be on the current device, cuda:0"):
                call(a.q)
        a = _args()
        for f in fields:
            setattr(a, f, _Elsewhere(getattr(a, f), 1 if f == "sl" else 0))
        for name in ("write", "bounds", "select"):
            with pytest.raises(ValueError, match="seq_lens must be on the current device, cuda:0"):
                _calls(pa, a)[name]()
    finally:
        calls.bind(pa.PAError, pa._current_device, pa._raw_current_stream)


@pytest.mark.parametrize("field,value,names", [
    ("pool", torch.zeros(2, 6, 16, 2, 64, dtype=torch.int8), ["write", "decode", "bounds"]),
    ("pool", torch.zeros(2, 6, 32, 2, 64, dtype=torch.uint8), ["write", "decode", "bounds"]),
    ("pool16", torch.zeros(2, 6, 16, 2, 64), ["sparse"]),
    ("pool16", torch.zeros(2, 6, 16, 2, 64, dtype=torch.bfloat16), ["sparse"]),
    ("scales", torch.ones(2, 6, 3), ["write", "decode", "bounds"]),
    ("scales", torch.ones(2, 6, 2, dtype=torch.float64), ["write", "decode", "bounds"]),
    ("scales", torch.ones(2, 6, 4)[:, :, ::2], ["write", "decode", "bounds"]),
    ("scales", None, ["write", "decode"]),
    ("tables", torch.zeros(3, 2, dtype=torch.int64), CALLS),
    ("tables", torch.zeros(2, 2, dtype=torch.int32), CALLS),
    ("tables", torch.zeros(2, 3, dtype=torch.int32).t(), CALLS),
    ("sl", torch.ones(3), CALLS),
    ("sl", torch.ones(6, dtype=torch.int32)[::2], CALLS),
    ("qsl", torch.zeros(3, dtype=torch.int32), ["write", "bounds"]),
    ("key", torch.zeros(3, 2, 128, dtype=torch.float16)[..., :64], ["write"]),
    ("key", torch.zeros(3, 2, 64), ["write"]),
    ("key", torch.zeros(3, 64, 2, dtype=torch.float16).transpose(1, 2), ["write"]),
    ("q", torch.zeros(3, 4, 64), ["decode", "select", "sparse"]),
    ("q", torch.zeros(3, 4, 32, dtype=torch.float16), ["decode", "select", "sparse"]),
    ("q", torch.zeros(4, 3, 64, dtype=torch.float16).transpose(0, 1), ["decode", "select",
                                                                       "sparse"]),
    ("bounds", torch.zeros(6, 2, 64, 2, dtype=torch.int8), ["bounds", "select"]),
    ("bounds", torch.zeros(6, 2, 2, 64, dtype=torch.uint8), ["bounds", "select"]),
    ("bsc", torch.ones(6, 3), ["bounds", "select"]),
    ("lists", torch.zeros(3, 4, 2, dtype=torch.int32), ["select", "sparse"]),
    ("lists", torch.zeros(3, 2, 2, dtype=torch.int64), ["select", "sparse"]),
    ("lens", torch.zeros(4, dtype=torch.int32), ["select", "sparse"]),
])
def test_binding_checks_shapes(pa, field, value, names):
    for name in names:
        a = _args()
        setattr(a, field, value)
        with pytest.raises(ValueError) as e:
            _calls(pa, a)[name]()
        assert "CUDA" not in str(e.value), (name, e.value)


def test_a_broadcast_key_is_refused(pa):
    """A row stride of zero is no row stride."""
    a = _args()
    a.key = torch.zeros(1, 2, 64, dtype=torch.float16).expand(3, 2, 64)
    with pytest.raises(ValueError, match="contiguous rows"):
        _calls(pa, a)["write"]()


def test_what_is_no_tensor_is_refused(pa):
    for field, value in (("pool", None), ("pool", 7), ("sl", [1, 2, 3]), ("tables", "x")):
        a = _args()
        setattr(a, field, value)
        with pytest.raises((AttributeError, TypeError, ValueError)):
            _calls(pa, a)["write"]()
    with pytest.raises(ValueError, match="32 bits"):
        pa.pa_update_block_bounds(*[None] * 6, 2 ** 40, 1)
    with pytest.raises(TypeError):
        pa.pa_decode_fp8_block(*[None] * 6, "0.1", 16, 16, None)


def test_a_failed_call_raises_its_status(pa):
    """The C call's own refusal comes out as PAError (no launch: the workspace
    is too small)."""
    calls = pa._block_calls
    calls.bind(pa.PAError, lambda: 0, lambda device: 0)
    try:
        a = _args()
        for f in vars(a):
            if f != "bs":
                setattr(a, f, _Elsewhere(getattr(a, f), 0))
        with pytest.raises(pa.PAError) as e:
            _calls(pa, a)["select"]()
        assert e.value.status in (INVALID, WORKSPACE) and "pa_select_blocks" in str(e.value)
    finally:
        calls.bind(pa.PAError, pa._current_device, pa._raw_current_stream)
