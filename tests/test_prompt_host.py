"""Refusals of the rotary, prompt-attention and quantised paged-cache calls
before anything reaches a GPU, and the tables of turns."""
import math

import numpy as np
import pytest

torch = pytest.importorskip("torch")

FAKE = 1 << 20         # a 16-byte aligned address that is never followed
MB = 1 << 20


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


ROPE = dict(q=1 * MB, qs=1024, qo=2 * MB, qos=1024, heads=8, k=3 * MB, ks=256, ko=4 * MB, kos=256, kv=2, pos=FAKE, rows=3, table=FAKE,
            rot=64, form=0, amp=1.0, d=128, dtype=1, stream=None)
PROMPT = dict(q=1 * MB, qs=1024, rows=9, k=2 * MB, ks=256, v=3 * MB, vs=256, krows=20, heads=2, groups=4, d=128, dtype=1, qst=FAKE, kst=FAKE,
              n=2, scale=0.1, out=4 * MB, os=1024, stream=None)
WRITE = dict(k=FAKE, v=FAKE, ks=256, vs=256, slot=FAKE, rows=3, K=FAKE, V=FAKE, kscale=FAKE, vscale=FAKE, pages=8, heads=2, ps=16, d=128,
             dtype=3, stream=None)
READ = dict(K=FAKE, V=FAKE, kscale=FAKE, vscale=FAKE, pages=8, heads=2, ps=16, d=128, dtype=5, slot=FAKE, rows=3, k=1 * MB, ks=256, v=2 * MB,
            vs=256, stream=None)
ATTEND = dict(q=FAKE, qs=1024, seq=FAKE, pos=FAKE, rows=3, K=FAKE, V=FAKE, kscale=FAKE, vscale=FAKE, pages=8, heads=2, groups=4, ps=16, d=128,
              dtype=3, table=FAKE, n=2, width=20, scale=0.1, out=FAKE, os=1024, stream=None)


@pytest.mark.parametrize("change,frag", [
    (dict(dtype=2), "dtype"), (dict(d=96), "head_dim"), (dict(rows=-1), "rows"), (dict(heads=0), "heads"), (dict(kv=-1), "heads"),
    (dict(rows=1 << 27), "2^28"), (dict(heads=1 << 21, rows=1), "2^20"), (dict(rot=0), "rot_dim"), (dict(rot=63), "rot_dim"), (dict(rot=130), "rot_dim"),
    (dict(form=2), "form"), (dict(amp=float("nan")), "amplitude"), (dict(amp=1e39), "amplitude"), (dict(table=None), "table"),
    (dict(table=FAKE + 4), "table"), (dict(q=None), "non-NULL"), (dict(ko=None), "non-NULL"), (dict(pos=None), "non-NULL"),
    (dict(pos=FAKE + 2), "aligned"), (dict(k=3 * MB + 8), "aligned"), (dict(qs=1023), "apart"), (dict(kos=260), "boundaries"),
    (dict(qo=1 * MB + 256), "overlaps"), (dict(qo=1 * MB, qos=2048), "overlaps"), (dict(ko=1 * MB), "overlaps"), (dict(ko=2 * MB), "overlaps"),
])
def test_rope_refuses(L, change, frag):
    _refused(L, "h2o_rope", ROPE, change, frag)


def test_rope_takes_slices_of_one_buffer(L):
    # q, k (and v) side by side in rows of 1536 elements, turned in place or into other columns; nothing is launched for no rows,
    # so the columns are checked by a refusal that comes after
    fused = dict(ROPE, qs=1536, qos=1536, ks=1536, kos=1536, q=MB, qo=MB, k=MB + 2048, ko=MB + 2048)
    lib = L.lib()
    import os
    os.environ["H2O_FAULT"] = "launch"
    try:
        for change in (dict(), dict(ko=MB + 2048 + 512), dict(k=None, ko=None, kv=0)):
            rc = lib.h2o_rope(*dict(fused, **change).values())
            assert rc == L.H2O_ERR_CUDA, L.h2o_last_error()
        for change in (dict(ko=MB + 2048 + 256), dict(qo=MB + 512), dict(ko=MB + 512)):
            rc = lib.h2o_rope(*dict(fused, **change).values())
            assert rc == L.H2O_ERR_ARG and "overlaps" in L.h2o_last_error()
    finally:
        del os.environ["H2O_FAULT"]


@pytest.mark.parametrize("change,frag", [
    (dict(dtype=3), "dtype"), (dict(d=80), "head_dim"), (dict(rows=-1), "rows"), (dict(krows=-1), "rows"), (dict(heads=0), "kv_heads"),
    (dict(heads=65536), "kv_heads"), (dict(groups=0), "groups"), (dict(groups=17), "groups"), (dict(n=0), "requests"), (dict(n=16385), "requests"),
    (dict(rows=(1 << 24) + 1), "2^24"), (dict(krows=(1 << 24) + 1), "2^24"), (dict(rows=1 << 23, groups=16, heads=4), "2^28"),
    (dict(krows=1 << 24, heads=32), "2^28"), (dict(n=16384, heads=257, rows=1, krows=1, qs=257 * 512, os=257 * 512, ks=257 * 128, vs=257 * 128), "2^22"), (dict(scale=0.0), "scale"), (dict(scale=float("inf")), "scale"),
    (dict(scale=1e-60), "scale"), (dict(qst=None), "q_start"), (dict(kst=FAKE + 2), "k_start"), (dict(q=None), "non-NULL"), (dict(v=None), "non-NULL"),
    (dict(out=4 * MB + 8), "aligned"), (dict(qs=1000), "apart"), (dict(vs=257), "boundaries"), (dict(out=1 * MB), "overlaps"),
    (dict(out=2 * MB + 512), "overlaps"), (dict(out=3 * MB), "overlaps"),
])
def test_prompt_refuses(L, change, frag):
    _refused(L, "h2o_prompt_attend", PROMPT, change, frag)


POOL = [
    (dict(K=None), "non-NULL"), (dict(vscale=None), "non-NULL"), (dict(V=FAKE + 8), "aligned"), (dict(kscale=FAKE + 4), "aligned"), (dict(dtype=1), "dtype"),
    (dict(dtype=7), "dtype"), (dict(dtype=11), "dtype"), (dict(d=96), "head_dim"), (dict(ps=8), "page_size"), (dict(pages=0), "num_pages"),
    (dict(heads=0), "kv_heads"), (dict(heads=65536), "kv_heads"), (dict(pages=1 << 27), "2^31"),
]


@pytest.mark.parametrize("change,frag", POOL + [
    (dict(rows=-1), "rows"), (dict(rows=1 << 28), "2^28"), (dict(k=None), "non-NULL"), (dict(slot=None), "non-NULL"), (dict(slot=FAKE + 2), "aligned"),
    (dict(v=FAKE + 8), "aligned"), (dict(ks=255), "apart"), (dict(vs=260), "boundaries"),
])
def test_quantised_rows_refuse(L, change, frag):
    _refused(L, "h2o_page_quant_write", WRITE, change, frag)
    _refused(L, "h2o_page_quant_read", READ, change, frag)


def test_quantised_read_refuses_keys_over_values(L):
    _refused(L, "h2o_page_quant_read", READ, dict(v=1 * MB + 256), "overlaps")


@pytest.mark.parametrize("change,frag", POOL + [
    (dict(rows=-1), "rows"), (dict(groups=0), "groups"), (dict(groups=17), "groups"), (dict(n=0), "requests"), (dict(width=0), "table_width"),
    (dict(width=16385), "table_width"), (dict(scale=0.0), "scale"), (dict(rows=1 << 22), "2^24"), (dict(table=None), "table"), (dict(q=None), "non-NULL"),
    (dict(pos=None), "non-NULL"), (dict(table=FAKE + 2), "aligned"), (dict(out=FAKE + 8), "aligned"), (dict(qs=1000), "apart"), (dict(os=1028), "boundaries"),
    (dict(out=FAKE + 256), "overlaps"),
])
def test_quantised_attend_refuses(L, change, frag):
    _refused(L, "h2o_page_quant_attend", ATTEND, change, frag)


def test_no_rows_is_no_work(L):
    for name, base in (("h2o_rope", ROPE), ("h2o_prompt_attend", PROMPT), ("h2o_page_quant_write", WRITE), ("h2o_page_quant_read", READ),
                       ("h2o_page_quant_attend", ATTEND)):
        assert getattr(L.lib(), name)(*dict(base, rows=0).values()) == L.H2O_OK


def test_tables(L):
    pair = np.arange(32)
    f = 10000.0 ** (-pair / 32)
    turns = lambda t: np.asarray(t, np.float64) * 2.0 ** -64 * 2 * math.pi    # noqa: E731
    # pow and the division are off by a few of fp64's half steps
    near = lambda t, want: np.all(np.abs(turns(t) - want) <= 8 * 2.0 ** -53 * want + 2.0 ** -60)    # noqa: E731
    assert near(L.h2o_rope_table(64), f)
    assert near(L.h2o_rope_table(64, kind=L.H2O_ROPE_LINEAR, factor=4.0), f / 4)
    raised = L.h2o_rope_table(64, kind=L.H2O_ROPE_BASE, factor=4.0)
    assert turns(raised)[0] == pytest.approx(1.0, rel=1e-14) and turns(raised)[-1] == pytest.approx(f[-1] / 4, rel=1e-13)
    parts = turns(L.h2o_rope_table(64, kind=L.H2O_ROPE_PARTS, factor=8.0, original_len=4096.0, low=1.0, high=32.0))
    t = 4096 * f / (2 * math.pi)
    g = np.clip((t - 1) / 31, 0, 1)
    assert np.allclose(parts, f * ((1 - g) / 8 + g), rtol=1e-13, atol=0)
    assert (g == 1).any() and (g == 0).any() and ((g > 0) & (g < 1)).any()
    assert L.h2o_rope_table(2, base=1.0).tolist() == [round(2.0 ** 64 / (2 * math.pi))]


@pytest.mark.parametrize("args,frag", [
    ((63,), "rot_dim"), ((0,), "rot_dim"), ((130,), "rot_dim"), ((64, 0.5), "base"), ((64, float("inf")), "base"), ((64, 1e4, 4), "kind"), ((64, 1e4, -1), "kind"),
    ((64, 1e4, 1, 0.5), "factor"), ((64, 1e4, 2, float("nan")), "factor"), ((2, 1e4, 2, 4.0), "rot_dim"), ((64, 1e300, 2, 1e30), "range"),
    ((64, 1e4, 3, 4.0, 0.0, 1.0, 32.0), "original_len"), ((64, 1e4, 3, 4.0, 4096.0, 32.0, 32.0), "low"),
])
def test_table_refuses(L, args, frag):
    with pytest.raises(L.H2OError, match=frag) as e:
        L.h2o_rope_table(*args)
    assert e.value.code == L.H2O_ERR_ARG


def test_binding_wants_fitting_tensors(L):
    q = torch.zeros(3, 8, 128, dtype=torch.bfloat16)
    k = torch.zeros(3, 2, 128, dtype=torch.bfloat16)
    i32 = lambda n: torch.zeros(n, dtype=torch.int32)    # noqa: E731
    with pytest.raises(ValueError, match="GPU"):
        L.h2o_rope(q, k, i32(3), torch.zeros(32, dtype=torch.int64), 0, 1.0, q, k)
    with pytest.raises(TypeError, match="q must be"):
        L.h2o_rope(q.half(), k, i32(3), torch.zeros(32, dtype=torch.int64), 0, 1.0, q, k)
    with pytest.raises(ValueError, match="GPU"):
        L.h2o_prompt_attend(q, k, k, i32(2), None, 0.1, q)
    with pytest.raises(TypeError, match="q must be"):
        L.h2o_prompt_attend(None, k, k, i32(2), None, 0.1, q)
    codes, scales = torch.zeros(4, 2, 16, 128, dtype=torch.int8), torch.zeros(4, 2, 16)
    with pytest.raises(TypeError, match="int8 or uint8"):
        L.h2o_page_quant_write(k, k, i32(3), codes.float(), codes, scales, scales)
    with pytest.raises(ValueError, match="GPU"):
        L.h2o_page_quant_read(codes, codes, scales, scales, i32(3), k, k)
    with pytest.raises(ValueError, match="codes"):
        L.h2o_page_quant_attend(q, i32(3), i32(3), codes[0], codes[0], scales, scales, torch.zeros(1, 4, dtype=torch.int32), 0.1, q)
