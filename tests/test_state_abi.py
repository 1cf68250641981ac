"""Host-side checks of linear attention and of fork, extend and compact: every refusal
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


class Pool(ctypes.Structure):
    _fields_ = [("data", P), ("block_bytes", I64), ("planes", ctypes.c_int32)]


def pools(*of):
    return (Pool * max(1, len(of)))(*[Pool(*x) for x in of])


def _caller(pa, name, spec):
    fn = getattr(ctypes.CDLL(pa.lib_path()), name)
    fn.restype = I
    fn.argtypes = [t for _, t, _ in spec]

    def call(**kw):
        values = {n: v for n, _, v in spec}
        assert set(kw) <= set(values)
        values.update(kw)
        return fn(*[values[n] for n, _, _ in spec])
    return call


HEAD = [("out", P, FAKE), ("q", P, FAKE), ("k", P, FAKE), ("v", P, FAKE), ("decay", P, FAKE),
        ("dstride", I64, 2), ("states", P, FAKE), ("src", P, FAKE), ("dst", P, FAKE)]
SIZES = [("H", I, 4), ("Hkv", I, 2), ("D", I, 64), ("NS", I, 8)]
STRIDES = [("qs", I64, 256), ("ks", I64, 128), ("vs", I64, 128), ("scale", F, 0.1), ("dtype", I, 0)]
DECODE = [*HEAD, ("B", I, 4), *SIZES, *STRIDES, ("stream", P, None)]
PREFILL = [*HEAD, ("starts", P, FAKE), ("B", I, 4), ("T", I, 40), ("most", I, 20), *SIZES, *STRIDES,
           ("ws", P, FAKE), ("wb", SZ, 1 << 30), ("stream", P, None)]

LINEAR = [(dict(B=-1), INVALID), (dict(H=0), INVALID), (dict(Hkv=0), INVALID), (dict(H=3), INVALID),
          (dict(D=0), INVALID), (dict(NS=0), INVALID), (dict(scale=float("nan")), INVALID),
          (dict(scale=float("inf")), INVALID), (dict(D=96), UNSUPPORTED), (dict(dtype=2), UNSUPPORTED),
          (dict(B=65536), UNSUPPORTED), (dict(qs=255), INVALID), (dict(qs=260), INVALID),
          (dict(ks=120), INVALID), (dict(vs=129), INVALID), (dict(dstride=1), INVALID),
          (dict(dstride=-2), INVALID), (dict(out=0), INVALID), (dict(q=0), INVALID),
          (dict(k=0), INVALID), (dict(v=0), INVALID), (dict(decay=0), INVALID),
          (dict(states=0), INVALID), (dict(src=0), INVALID), (dict(dst=0), INVALID),
          (dict(out=FAKE + 8), INVALID), (dict(q=FAKE + 8), INVALID), (dict(k=FAKE + 4), INVALID),
          (dict(v=FAKE + 2), INVALID), (dict(decay=FAKE + 2), INVALID),
          (dict(states=FAKE + 4), INVALID), (dict(src=FAKE + 1), INVALID),
          (dict(dst=FAKE + 2), INVALID)]


@pytest.mark.parametrize("kw,status", LINEAR)
def test_linear_decode_refusals(pa, kw, status):
    assert _caller(pa, "pa_linear_decode", DECODE)(**kw) == status


@pytest.mark.parametrize("kw,status", LINEAR + [
    (dict(T=-1), INVALID), (dict(most=-1), INVALID), (dict(starts=0), INVALID),
    (dict(starts=FAKE + 2), INVALID), (dict(ws=0), WORKSPACE), (dict(ws=FAKE + 16), WORKSPACE),
    (dict(wb=255), WORKSPACE), (dict(T=1 << 20, most=1 << 20, wb=1 << 20), WORKSPACE)])
def test_linear_prefill_refusals(pa, kw, status):
    assert _caller(pa, "pa_linear_prefill", PREFILL)(**kw) == status


TABLES = [("tables", P, FAKE), ("lens", P, 2 * FAKE), ("refs", P, 3 * FAKE)]
OUT = [("tables_out", P, 4 * FAKE), ("lens_out", P, 5 * FAKE), ("refs_out", P, 6 * FAKE)]
COUNTS = [("NB", I, 100), ("MB", I, 10), ("bs", I, 16)]
FORK = [*OUT, *TABLES, ("parents", P, 7 * FAKE), ("R", I, 4), ("RO", I, 4), *COUNTS, ("stream", P, None)]
EXTEND = [*OUT, ("slots", P, 8 * FAKE), ("info", P, 9 * FAKE), *TABLES, ("new", P, 7 * FAKE),
          ("pools", P, None), ("np", I, 0), ("R", I, 4), ("T", I, 9), *COUNTS, ("ws", P, 16 * FAKE),
          ("wb", SZ, 1 << 20), ("stream", P, None)]
COMPACT = [OUT[0], OUT[2], ("ids", P, 8 * FAKE), ("info", P, 9 * FAKE), *TABLES, ("pools", P, None),
           ("np", I, 0), ("R", I, 4), *COUNTS, ("ws", P, 16 * FAKE), ("wb", SZ, 1 << 20),
           ("stream", P, None)]

BOOKS = [(dict(R=-1), INVALID), (dict(NB=0), INVALID), (dict(MB=0), INVALID), (dict(bs=0), INVALID),
         (dict(bs=-16), INVALID), (dict(R=65536), UNSUPPORTED), (dict(NB=(1 << 29) + 1), UNSUPPORTED),
         (dict(MB=1 << 20, bs=1 << 12), UNSUPPORTED), (dict(MB=1 << 27, bs=1), UNSUPPORTED),
         (dict(tables=0), INVALID), (dict(lens=0), INVALID), (dict(refs=0), INVALID),
         (dict(tables_out=0), INVALID), (dict(refs_out=0), INVALID), (dict(tables=FAKE + 2), INVALID),
         (dict(refs=3 * FAKE + 1), INVALID), (dict(refs_out=6 * FAKE + 2), INVALID),
         # outputs that overlap their inputs but are not they
         (dict(tables_out=FAKE + 40), INVALID), (dict(tables_out=FAKE - 40), INVALID),
         (dict(refs_out=3 * FAKE + 396), INVALID), (dict(refs_out=3 * FAKE - 4), INVALID)]


@pytest.mark.parametrize("kw,status", BOOKS + [
    (dict(RO=-1), INVALID), (dict(RO=65536), UNSUPPORTED), (dict(parents=0), INVALID),
    (dict(parents=7 * FAKE + 1), INVALID), (dict(lens_out=0), INVALID),
    # rows trade places: not in place
    (dict(tables_out=FAKE), INVALID), (dict(lens_out=2 * FAKE), INVALID),
    (dict(lens_out=2 * FAKE + 12), INVALID)])
def test_fork_refusals(pa, kw, status):
    assert _caller(pa, "pa_fork_sequences", FORK)(**kw) == status


POOLS = [(dict(np=-1), INVALID), (dict(np=1), INVALID),
         (dict(np=1, pools=pools((0, 16, 2))), INVALID), (dict(np=1, pools=pools((FAKE, 0, 2))), INVALID),
         (dict(np=1, pools=pools((FAKE, 16, 0))), INVALID),
         (dict(np=257, pools=pools(*[(FAKE, 16, 2)] * 257)), UNSUPPORTED),
         (dict(np=1, pools=pools((FAKE, 1 << 50, 2))), UNSUPPORTED),
         (dict(np=2, pools=pools((FAKE, 16, 2), (FAKE, -4, 1))), INVALID),
         (dict(ws=0), WORKSPACE), (dict(ws=16 * FAKE + 64), WORKSPACE), (dict(wb=100), WORKSPACE)]


@pytest.mark.parametrize("kw,status", BOOKS + POOLS + [
    (dict(T=-1), INVALID), (dict(slots=0), INVALID), (dict(slots=8 * FAKE + 4), INVALID),
    (dict(info=0), INVALID), (dict(new=0), INVALID), (dict(lens_out=0), INVALID),
    (dict(lens_out=2 * FAKE + 4), INVALID)])
def test_extend_refusals(pa, kw, status):
    assert _caller(pa, "pa_extend_sequences", EXTEND)(**kw) == status


@pytest.mark.parametrize("kw,status", BOOKS + POOLS + [
    (dict(ids=0), INVALID), (dict(info=0), INVALID), (dict(ids=3 * FAKE), INVALID),
    (dict(ids=6 * FAKE + 4), INVALID)])
def test_compact_refusals(pa, kw, status):
    assert _caller(pa, "pa_compact_blocks", COMPACT)(**kw) == status


# Sizes of the arrays of FORK, EXTEND and COMPACT as they stand above, in bytes.
SPANS = {"tables": 160, "lens": 16, "refs": 400, "tables_out": 160, "lens_out": 16, "refs_out": 400,
         "parents": 16, "new": 16, "slots": 72, "info": 8, "ids": 400}
MAY_BE = {"tables_out": "tables", "lens_out": "lens", "refs_out": "refs"}


@pytest.mark.parametrize("name,spec,outs,ins", [
    ("pa_fork_sequences", FORK, ["tables_out", "lens_out", "refs_out"],
     ["tables", "lens", "refs", "parents"]),
    ("pa_extend_sequences", EXTEND, ["tables_out", "lens_out", "refs_out", "slots", "info"],
     ["tables", "lens", "refs", "new"]),
    ("pa_compact_blocks", COMPACT, ["tables_out", "refs_out", "ids", "info"],
     ["tables", "lens", "refs"])])
def test_outputs_on_other_arrays(pa, name, spec, outs, ins):
    """An output that lies on any other array, by its first bytes or its last, is refused,
    but for the input that it may be."""
    call = _caller(pa, name, spec)
    at = {n: v for n, _, v in spec}
    both = [(o, x) for o in outs for x in ins + outs if x != o] + \
        ([(o, "ws") for o in outs] + [("ws", x) for x in ins] if "ws" in at else [])
    for out, other in both:
        if out == "ws":
            assert call(ws=at[other]) == INVALID, (out, other)
            continue
        least = 256 if other == "ws" else SPANS[other]
        for place in (at[other] + least - 8, at[other] - SPANS[out] + 8, at[other]):
            if place == at[other] and MAY_BE.get(out) == other and name != "pa_fork_sequences":
                continue
            if place == at[other] and (out, other) == ("refs_out", "refs"):
                continue
            assert call(**{out: place}) == INVALID, (out, other, place - at[other])


def test_nothing_to_do_is_ok(pa):
    assert _caller(pa, "pa_linear_decode", DECODE)(B=0) == 0
    assert _caller(pa, "pa_linear_prefill", PREFILL)(B=0) == 0


def test_workspace_sizes(pa):
    size = pa.pa_linear_prefill_workspace_size
    assert size(16, 20000, 2000, 32, 128) == 256          # many chains: nothing to join
    assert size(1, 131072, 131072, 8, 128) > 64 * 8 * 128 * 128 * 4
    assert size(-1, 10, 10, 8, 128) == 0 and size(1, 10, 10, 0, 128) == 0
    assert size(1, -1, 10, 8, 128) == 0 and size(1, 10, -1, 8, 128) == 0
    for b, t, most in ((1, 131072, 131072), (1, 129, 129), (7, 30000, 9000), (300, 500000, 300000),
                       (2, 1 << 30, 1 << 30), (1, 2 ** 31 - 1, 2 ** 31 - 1)):
        for hkv in (1, 2, 5, 8, 32, 200, 1216, 1217):
            states = 1216 + (b + 1) * hkv
            assert 0 < size(b, t, most, hkv, 64) <= states * (64 * 64 * 4 + 4) + 255
    size = pa.pa_sequences_workspace_size
    assert size(0, 1) > 0 and size(100, 5000) >= 4 * (3 * 5000 + 6 * 100)
    assert size(-1, 10) == 0 and size(1, 0) == 0 and size(65536, 10) == 0


# ---------------------------------------------------------------------------
# The binding
# ---------------------------------------------------------------------------
def _args(b=3, h=4, hkv=2, d=64, t=9, nb=6, mb=2):
    i32 = dict(dtype=torch.int32)
    half = dict(dtype=torch.float16)
    return types.SimpleNamespace(
        q=torch.zeros(b, h, d, **half), k=torch.zeros(b, hkv, d, **half),
        v=torch.zeros(b, hkv, d, **half), g=torch.zeros(b, hkv), states=torch.zeros(8, hkv, d, d),
        src=torch.zeros(b, **i32), dst=torch.zeros(b, **i32), starts=torch.arange(b + 1, **i32),
        ws=torch.zeros(64, dtype=torch.uint8), tables=torch.zeros(b, mb, **i32),
        lens=torch.ones(b, **i32), refs=torch.zeros(nb, **i32), tout=torch.zeros(b, mb, **i32),
        lout=torch.zeros(b, **i32), rout=torch.zeros(nb, **i32), parents=torch.zeros(b, **i32),
        new=torch.zeros(b, **i32), slots=torch.zeros(t, dtype=torch.int64), info=torch.zeros(2, **i32),
        ids=torch.zeros(nb, **i32), pool=torch.zeros(2, nb, 16, hkv, d, **half))


def _calls(pa, a):
    return {
        "ldec": lambda: pa.pa_linear_decode(torch.empty(a.q.shape, dtype=a.q.dtype), a.q, a.k, a.v, a.g,
                                            a.states, a.src, a.dst, 0.1),
        "lpre": lambda: pa.pa_linear_prefill(torch.empty(a.q.shape, dtype=a.q.dtype), a.q, a.k, a.v, a.g,
                                             a.states, a.src, a.dst, a.starts, 0.1, 1, a.ws),
        "fork": lambda: pa.pa_fork_sequences(a.tout, a.lout, a.rout, a.tables, a.lens, a.refs, a.parents, 16),
        "extend": lambda: pa.pa_extend_sequences(a.tout, a.lout, a.rout, a.slots, a.info, a.tables, a.lens,
                                                 a.refs, a.new, [a.pool], 16, a.ws),
        "compact": lambda: pa.pa_compact_blocks(a.tout, a.rout, a.ids, a.info, a.tables, a.lens, a.refs,
                                                [a.pool], 16, a.ws),
    }


CALLS = ["ldec", "lpre", "fork", "extend", "compact"]
LIN, SEQ = CALLS[:2], CALLS[2:]


@pytest.mark.parametrize("name", CALLS)
def test_binding_wants_cuda_tensors(pa, name):
    with pytest.raises(ValueError, match="must be a CUDA tensor"):
        _calls(pa, _args())[name]()


@pytest.mark.parametrize("field,value,names", [
    ("q", torch.zeros(3, 4, 64), LIN),
    ("q", torch.zeros(3, 256, dtype=torch.float16), LIN),
    ("q", torch.zeros(3, 4, 128, dtype=torch.float16)[..., :64], LIN),
    ("q", torch.zeros(3, 64, 4, dtype=torch.float16).transpose(1, 2), LIN),
    ("q", torch.zeros(1, 4, 64, dtype=torch.float16).expand(3, 4, 64), LIN),
    ("k", torch.zeros(3, 2, 64, dtype=torch.bfloat16), LIN),
    ("k", torch.zeros(2, 2, 64, dtype=torch.float16), LIN),
    ("v", torch.zeros(3, 1, 64, dtype=torch.float16), LIN),
    ("v", torch.zeros(3, 2, 32, dtype=torch.float16), LIN),
    ("g", torch.zeros(3, 2, dtype=torch.float64), LIN),
    ("g", torch.zeros(3, 4), LIN),
    ("g", torch.zeros(2, 2), LIN),
    ("g", torch.zeros(3, 4)[:, ::2], LIN),
    ("g", torch.zeros(()), LIN),
    ("states", torch.zeros(8, 2, 64, 32), LIN),
    ("states", torch.zeros(8, 2, 64, 64, dtype=torch.float16), LIN),
    ("states", torch.zeros(8, 2, 64, 128)[..., ::2], LIN),
    ("states", torch.zeros(8, 4, 64, 64), LIN),
    ("src", torch.zeros(3, dtype=torch.int64), LIN),
    ("src", torch.zeros(2, dtype=torch.int32), LIN),
    ("dst", torch.zeros(6, dtype=torch.int32)[::2], LIN),
    ("dst", torch.zeros(2, dtype=torch.int32), LIN),
    ("starts", torch.zeros(3, dtype=torch.int32), ["lpre"]),
    ("tables", torch.zeros(3, 2, dtype=torch.int64), SEQ),
    ("tables", torch.zeros(2, 3, dtype=torch.int32).t(), SEQ),
    ("lens", torch.ones(2, dtype=torch.int32), SEQ),
    ("refs", torch.zeros(6, dtype=torch.int64), SEQ),
    ("refs", torch.zeros(12, dtype=torch.int32)[::2], SEQ),
    ("tout", torch.zeros(3, 3, dtype=torch.int32), SEQ),
    ("tout", torch.zeros(4, 2, dtype=torch.int32), SEQ),
    ("rout", torch.zeros(5, dtype=torch.int32), SEQ),
    ("lout", torch.zeros(4, dtype=torch.int32), ["fork", "extend"]),
    ("parents", torch.zeros(3), ["fork"]),
    ("new", torch.zeros(4, dtype=torch.int32), ["extend"]),
    ("slots", torch.zeros(9, dtype=torch.int32), ["extend"]),
    ("info", torch.zeros(3, dtype=torch.int32), ["extend", "compact"]),
    ("ids", torch.zeros(5, dtype=torch.int32), ["compact"]),
])
def test_binding_checks_shapes(pa, field, value, names):
    for name in names:
        a = _args()
        setattr(a, field, value)
        with pytest.raises(ValueError) as e:
            _calls(pa, a)[name]()
        assert "CUDA" not in str(e.value), (name, e.value)


class _Elsewhere:
    """A CPU tensor that says it lies on another device."""

    def __init__(self, tensor, device):
        self.tensor, self.device = tensor, device

    def get_device(self):
        return self.device

    def __getattr__(self, name):
        return getattr(self.tensor, name)


def test_binding_wants_the_current_device(pa):
    calls = pa._block_calls
    calls.bind(pa.PAError, lambda: 0, lambda device: 0)
    try:
        fields = list(vars(_args()))
        for bad, names in (("states", LIN), ("refs", SEQ), ("pool", ["extend", "compact"]),
                           ("ws", ["lpre", "extend", "compact"])):
            a = _args()
            for f in fields:
                setattr(a, f, _Elsewhere(getattr(a, f), 1 if f == bad else 0))
            for name in names:
                if name in LIN:  # out is made by the test
                    call = getattr(calls, "linear_decode" if name == "ldec" else "linear_prefill")
                    first = [a.q, a.q, a.k, a.v, a.g, a.states, a.src, a.dst]
                    last = [0.1, None] if name == "ldec" else [a.starts, a.ws, 0.1, 1, None]
                    with pytest.raises(ValueError, match="current device"):
                        call(*first, *last)
                else:
                    with pytest.raises(ValueError, match="current device"):
                        _calls(pa, a)[name]()
    finally:
        calls.bind(pa.PAError, pa._current_device, pa._raw_current_stream)


@pytest.mark.parametrize("pool", [
    torch.zeros(6), torch.zeros(2, 5, 4), torch.zeros(2, 6, 4)[..., ::2], torch.zeros(2, 6, 0), 3, None])
def test_binding_checks_pools(pa, pool):
    calls = pa._block_calls
    calls.bind(pa.PAError, lambda: 0, lambda device: 0)
    try:
        a = _args()
        for f in vars(a):
            if f != "pool":
                setattr(a, f, _Elsewhere(getattr(a, f), 0))
        a.pool = _Elsewhere(pool, 0) if isinstance(pool, torch.Tensor) else pool
        for name in ("extend", "compact"):
            with pytest.raises((ValueError, AttributeError, TypeError)):
                _calls(pa, a)[name]()
        # the pools themselves are no list
        with pytest.raises((TypeError, ValueError)):
            pa.pa_compact_blocks(a.tout, a.rout, a.ids, a.info, a.tables, a.lens, a.refs, 7, 16, a.ws)
    finally:
        calls.bind(pa.PAError, pa._current_device, pa._raw_current_stream)


def test_a_list_of_pools_that_changes_meanwhile(pa):
    """The pools are those that the list held when the call was made."""
    calls = pa._block_calls
    calls.bind(pa.PAError, lambda: 0, lambda device: 0)
    try:
        a = _args()
        for f in vars(a):
            setattr(a, f, _Elsewhere(getattr(a, f), 0))
        seen = []

        class Pool(_Elsewhere):
            def get_device(self):
                seen.append(len(pools))
                pools.clear()
                return 0

        pools = [Pool(torch.zeros(2, 6, 16), 0) for _ in range(5)]
        with pytest.raises(pa.PAError) as e:  # the workspace is too small: no launch
            pa.pa_compact_blocks(a.tout, a.rout, a.ids, a.info, a.tables, a.lens, a.refs, pools, 16, a.ws)
        assert e.value.status in (INVALID, WORKSPACE)
        assert seen == [5, 0, 0, 0, 0]
    finally:
        calls.bind(pa.PAError, pa._current_device, pa._raw_current_stream)


def test_a_failed_call_raises_its_status(pa):
    """The C call's own refusal comes out as PAError (no launch: the workspace is too
    small)."""
    calls = pa._block_calls
    calls.bind(pa.PAError, lambda: 0, lambda device: 0)
    try:
        a = _args()
        for f in vars(a):
            setattr(a, f, _Elsewhere(getattr(a, f), 0))
        for name in ("extend", "compact"):
            with pytest.raises(pa.PAError) as e:
                _calls(pa, a)[name]()
            assert e.value.status in (INVALID, WORKSPACE)
    finally:
        calls.bind(pa.PAError, pa._current_device, pa._raw_current_stream)
