"""Refusals of the paged-cache calls, before anything reaches a GPU: the C
calls with made-up pointers, and the binding with tensors that do not fit."""
import pytest

torch = pytest.importorskip("torch")

FAKE = 1 << 20         # a 16-byte aligned address that is never followed


@pytest.fixture(scope="module")
def L():
    from kv_cache_eviction_h2o_gb300 import build as b
    b.build()
    from kv_cache_eviction_h2o_gb300 import binding
    return binding


def _refused(L, name, base, change, frag, code=None):
    args = dict(base, **change)
    rc = getattr(L.lib(), name)(*args.values())
    assert rc == (L.H2O_ERR_ARG if code is None else code), (change, rc)
    assert frag in L.h2o_last_error(), (change, L.h2o_last_error())


TABLES = dict(before=FAKE, new=FAKE, n=4, free=FAKE, n_free=8, ps=16, table=FAKE, width=4, after=FAKE, start=FAKE, seq=FAKE,
              pos=FAKE, slot=FAKE, cap=8, status=FAKE, stream=None)
WRITE = dict(k=FAKE, v=FAKE, ks=256, vs=256, slot=FAKE, rows=3, K=FAKE, V=FAKE, bounds=FAKE, pages=8, heads=2, ps=16, d=128,
             dtype=1, stream=None)
ATTEND = dict(q=FAKE, qs=1024, seq=FAKE, pos=FAKE, rows=3, K=FAKE, V=FAKE, bounds=FAKE, pages=8, heads=2, groups=4, ps=16,
              d=128, dtype=1, table=FAKE, n=2, width=20, budget=8, recent=2, scale=0.1, out=FAKE, os=1024, picked=None, stream=None)
PREFIX = dict(q=FAKE, qs=1024, seq=FAKE, pos=FAKE, rows=3, K=FAKE, V=FAKE, pages=8, heads=2, groups=4, ps=16, d=128, dtype=1,
              pt=FAKE, plen=40, table=FAKE, n=2, width=20, scale=0.1, out=FAKE, os=1024, work=FAKE, nwork=1 << 40, stream=None)


@pytest.mark.parametrize("change,frag", [
    (dict(n=0), "requests"), (dict(n=16385), "requests"), (dict(n_free=-1), "n_free"), (dict(cap=-1), "rows_cap"), (dict(cap=(1 << 30) + 1), "rows_cap"),
    (dict(ps=48), "page_size"), (dict(width=0), "table_width"), (dict(width=16385), "table_width"), (dict(before=None), "non-NULL"),
    (dict(free=None), "non-NULL"), (dict(slot=None), "non-NULL"), (dict(status=None), "non-NULL"), (dict(seq=FAKE + 2), "aligned"),
])
def test_tables_refuses(L, change, frag):
    _refused(L, "h2o_page_tables", TABLES, change, frag)


@pytest.mark.parametrize("change", [
    dict(after=1 << 20), dict(start=(1 << 20) + 12), dict(table=(1 << 20) - 4 * 4 * 4 + 4), dict(status=2 << 20), dict(slot=(3 << 20) - 28),
    dict(seq=(3 << 20) + 28), dict(pos=2 << 20),
])
def test_tables_refuses_outputs_over_inputs(L, change):
    apart = dict(TABLES, **{k: (i + 1) << 20 for i, k in enumerate(("before", "new", "free", "table", "after", "start", "seq", "pos",
                                                                  "slot", "status"))})
    _refused(L, "h2o_page_tables", apart, change, "overlaps")


def test_prefixes_beyond_its_range_are_refused(L):
    for n in ((1 << 30) + 1, (1 << 31) - 1):
        _refused(L, "h2o_prefix_attend", PREFIX, dict(plen=n), "prefix_len")
        with pytest.raises(L.H2OError):
            L.h2o_prefix_work_bytes(4, 8, 4, 128, n, L.H2O_BF16)
    for dtype in (L.H2O_BF16, L.H2O_F32):
        assert L.h2o_prefix_work_bytes(4, 8, 4, 128, 1 << 30, dtype) > 0


POOL = [
    (dict(K=None), "non-NULL"), (dict(V=FAKE + 8), "aligned"), (dict(dtype=8), "dtype"), (dict(d=96), "head_dim"),
    (dict(ps=8), "page_size"), (dict(ps=256), "page_size"), (dict(pages=0), "num_pages"), (dict(heads=0), "kv_heads"),
    (dict(heads=65536), "kv_heads"), (dict(pages=1 << 27), "2^31"),
]


@pytest.mark.parametrize("change,frag", POOL + [
    (dict(bounds=None), "bounds"), (dict(rows=-1), "rows"), (dict(k=None), "non-NULL"), (dict(slot=FAKE + 2), "aligned"),
    (dict(ks=255), "apart"), (dict(vs=260), "boundaries"), (dict(v=FAKE + 2), "aligned"),
])
def test_write_refuses(L, change, frag):
    _refused(L, "h2o_page_write", WRITE, change, frag)


ROWS = [
    (dict(rows=-1), "rows"), (dict(groups=0), "groups"), (dict(groups=17), "groups"), (dict(n=0), "requests"),
    (dict(width=0), "table_width"), (dict(width=16385), "table_width"), (dict(scale=0.0), "scale"), (dict(scale=float("nan")), "scale"),
    (dict(scale=float("inf")), "scale"), (dict(rows=1 << 22), "2^24"), (dict(table=None), "table"), (dict(q=None), "non-NULL"),
    (dict(pos=None), "non-NULL"), (dict(table=FAKE + 2), "aligned"), (dict(out=FAKE + 8), "aligned"), (dict(qs=1000), "apart"),
    (dict(os=1028), "boundaries"),
]


@pytest.mark.parametrize("change,frag", POOL + ROWS + [
    (dict(recent=0), "recent"), (dict(recent=9), "recent"), (dict(bounds=None), "bounds"), (dict(bounds=FAKE + 4), "aligned"),
    (dict(width=8000, budget=4097), "4096"), (dict(picked=FAKE + 1), "aligned"),
])
def test_attend_refuses(L, change, frag):
    _refused(L, "h2o_page_attend", ATTEND, change, frag)


@pytest.mark.parametrize("change,frag", POOL + ROWS + [
    (dict(plen=-1), "prefix_len"), (dict(pt=None), "prefix_table"), (dict(pt=FAKE + 2), "prefix_table"), (dict(work=None), "work"),
    (dict(nwork=100), "work"), (dict(work=FAKE + 8), "work"),
])
def test_prefix_refuses(L, change, frag):
    _refused(L, "h2o_prefix_attend", PREFIX, change, frag)


def test_quantised_pools_are_unsupported(L):
    for flag in (L.H2O_KV8, L.H2O_KV4):
        for name, base in (("h2o_page_write", WRITE), ("h2o_page_attend", ATTEND), ("h2o_prefix_attend", PREFIX)):
            _refused(L, name, base, dict(dtype=1 | flag), "not supported", L.H2O_ERR_UNSUPPORTED)


def test_no_rows_is_no_work(L):
    # nothing is launched, so the made-up addresses are never used
    for name, base in (("h2o_page_write", WRITE), ("h2o_page_attend", ATTEND), ("h2o_prefix_attend", PREFIX)):
        assert getattr(L.lib(), name)(*dict(base, rows=0).values()) == L.H2O_OK


def test_workspace_size(L):
    a = L.h2o_prefix_work_bytes(64, 8, 4, 128, 1000, L.H2O_BF16)
    assert a >= 64 * 8 * 4 * (128 * 4 + 8)
    assert L.h2o_prefix_work_bytes(64, 8, 4, 128, 0, L.H2O_BF16) > 0
    assert L.h2o_prefix_work_bytes(0, 8, 4, 128, 1000, L.H2O_F32) > 0
    for bad in ((-1, 8, 4, 128, 10, 1), (4, 0, 4, 128, 10, 1), (4, 8, 17, 128, 10, 1), (4, 8, 4, 96, 10, 1), (4, 8, 4, 128, -1, 1),
                (4, 8, 4, 128, 10, 3), (1 << 24, 2, 1, 128, 10, 1)):
        with pytest.raises(L.H2OError) as e:
            L.h2o_prefix_work_bytes(*bad)
        assert e.value.code == L.H2O_ERR_ARG


def test_binding_wants_gpu_tensors_of_fitting_shapes(L):
    K = torch.zeros(4, 2, 16, 64)
    i = torch.zeros(3, dtype=torch.int32)
    with pytest.raises(ValueError, match="GPU"):
        L.h2o_page_write(torch.zeros(3, 2, 64), torch.zeros(3, 2, 64), i, K, K, torch.zeros(4, 2, 2, 64))
    with pytest.raises(ValueError, match="GPU"):
        L.h2o_page_tables(i, i, i, 16, torch.zeros(3, 2, dtype=torch.int32), i, torch.zeros(4, dtype=torch.int32), i, i, i, i)
    with pytest.raises(TypeError, match="dtype"):
        L.h2o_page_write(i, i, i, K.half(), K.half(), K)
    with pytest.raises(ValueError, match="pages"):
        L.h2o_page_write(i, i, i, K[0], K[0], K)
    cpu = -1               # get_device() of a CPU tensor
    with pytest.raises(ValueError, match="shape"):
        L._tensor(i, "slot", torch.int32, (4,), cpu)
    with pytest.raises(TypeError, match="dtype"):
        L._tensor(i.long(), "slot", torch.int32, (3,), cpu)
    with pytest.raises(ValueError, match="contiguous"):
        L._tensor(torch.zeros(3, 2, dtype=torch.int32).t(), "table", torch.int32, (2, 3), cpu)
    wide = torch.zeros(5, 3 * 8, 64)
    assert L._head_rows(wide[:, 8:16], "k", torch.float32, (5, 8, 64), cpu) == (wide.data_ptr() + 8 * 64 * 4, 24 * 64)
    with pytest.raises(ValueError, match="contiguous heads"):
        L._head_rows(wide[:, ::3], "k", torch.float32, (5, 8, 64), cpu)
    with pytest.raises(ValueError, match="contiguous heads"):
        L._head_rows(wide[..., ::2], "k", torch.float32, (5, 24, 32), cpu)


class _Gpu:
    """What the binding asks of a tensor, as one on cuda:0 would answer; a CPU tensor gives the shapes."""

    def __init__(self, x):
        self.x, self.dtype, self.shape, self.device = x, x.dtype, x.shape, "cuda:0"

    def __getattr__(self, name):
        return getattr(self.x, name)

    def get_device(self):
        return 0


class _Lib:
    """Records the last argument, the stream, of each call."""

    def __init__(self):
        self.streams = {}

    def __getattr__(self, name):
        def call(*args):
            self.streams[name] = args[-1]
            return 0
        return call


def _all_calls(L, **stream):
    i32 = lambda *n: _Gpu(torch.zeros(*n, dtype=torch.int32))   # noqa: E731
    f = lambda *n: _Gpu(torch.zeros(*n))                        # noqa: E731
    K, V, B, q, out = f(4, 2, 16, 64), f(4, 2, 16, 64), f(4, 2, 2, 64), f(3, 4, 64), f(3, 4, 64)
    L.h2o_page_tables(i32(2), i32(2), i32(5), 16, i32(2, 3), i32(2), i32(3), i32(3), i32(3), i32(3), i32(4), **stream)
    L.h2o_page_write(f(3, 2, 64), f(3, 2, 64), i32(3), K, V, B, **stream)
    L.h2o_page_attend(q, i32(3), i32(3), K, V, B, i32(2, 3), 2, 1, 0.1, out, **stream)
    L.h2o_prefix_attend(q, i32(3), i32(3), K, V, i32(1), 16, i32(2, 3), 0.1, out, _Gpu(torch.zeros(64, dtype=torch.uint8)), **stream)


def test_without_a_stream_calls_run_on_the_current_one(L, monkeypatch):
    import types
    lib = _Lib()
    monkeypatch.setattr(L, "lib", lambda: lib)
    monkeypatch.setattr(L, "_types", None)
    monkeypatch.setattr(torch.cuda, "current_device", lambda: 0)
    monkeypatch.setattr(torch.cuda, "current_stream", lambda *a: types.SimpleNamespace(cuda_stream=77))
    _all_calls(L)
    assert len(lib.streams) == 4 and set(lib.streams.values()) == {77}
    _all_calls(L, stream=types.SimpleNamespace(cuda_stream=5))
    assert set(lib.streams.values()) == {5}
    _all_calls(L, stream=6)
    assert set(lib.streams.values()) == {6}


# rows of 1024 elements (2048 bytes), 3 of them; q at FAKE
@pytest.mark.parametrize("change,refused", [
    (dict(out=FAKE), False), (dict(out=FAKE, qs=1032, os=1032), False), (dict(out=FAKE + 3 * 2048), False), (dict(out=FAKE - 3 * 2048), False),
    (dict(out=FAKE + 2048, qs=2048, os=2048), False), (dict(out=FAKE - 2048, qs=2560, os=2560), False), (dict(out=FAKE + 4 * 2048, qs=2048, os=2048), True),
    (dict(out=FAKE + 16), True), (dict(out=FAKE + 2048), True), (dict(out=FAKE - 2048), True), (dict(out=FAKE + 2 * 2048 + 2032), True),
    (dict(out=FAKE, os=2048), True), (dict(out=FAKE + 2032, qs=2048, os=2048), True), (dict(out=FAKE - 2048 - 16, qs=2048, os=2048), True),
    (dict(out=FAKE, qs=1024, os=4096, rows=1), False), (dict(out=FAKE + 16, rows=1), True), (dict(out=FAKE + 2048, rows=1), False),
    (dict(out=FAKE + 16, rows=0), False),
])
@pytest.mark.parametrize("dtype", [0, 1])
def test_outputs_over_other_rows_of_q_are_refused(L, monkeypatch, change, refused, dtype):
    monkeypatch.setenv("H2O_FAULT", "launch")              # what is not refused stops before its launch
    change = dict(change, dtype=dtype)
    if dtype == 0:                                         # the same bytes
        change["d"] = 64
        for k in ("qs", "os"):
            change[k] = change.get(k, 1024) // 2
    for name, base in (("h2o_page_attend", ATTEND), ("h2o_prefix_attend", PREFIX)):
        base = dict(base, d=128)
        rc = getattr(L.lib(), name)(*dict(base, **change).values())
        if refused:
            assert rc == L.H2O_ERR_ARG and "overlaps" in L.h2o_last_error(), (change, rc)
        else:
            assert rc == (L.H2O_OK if change.get("rows") == 0 else L.H2O_ERR_CUDA), (change, rc, L.h2o_last_error())


def test_binding_refuses_pools_without_heads(L, monkeypatch):
    monkeypatch.setattr(L, "_types", None)
    monkeypatch.setattr(torch.cuda, "current_device", lambda: 0)
    monkeypatch.setattr(torch.cuda, "current_stream", lambda *a: None)
    K, B, q = (_Gpu(torch.zeros(*n)) for n in ((4, 0, 16, 64), (4, 0, 2, 64), (3, 4, 64)))
    i, table, work = (_Gpu(torch.zeros(*n, dtype=t)) for n, t in (((3,), torch.int32), ((2, 3), torch.int32), ((64,), torch.uint8)))
    with pytest.raises(ValueError, match="0 cache heads"):
        L.h2o_page_attend(q, i, i, K, K, B, table, 2, 1, 0.1, q)
    with pytest.raises(ValueError, match="0 cache heads"):
        L.h2o_prefix_attend(q, i, i, K, K, i, 16, table, 0.1, q, work)
    with pytest.raises(L.H2OError, match="non-NULL"):         # (an empty tensor has no memory)
        L.h2o_page_write(_Gpu(torch.zeros(3, 0, 64)), _Gpu(torch.zeros(3, 0, 64)), i, K, K, B)
