"""Host-side checks of the 4-bit pool and of kv_unpack: what the library and
the binding refuse before any launch.  Runs without a GPU."""
import ctypes

import pytest
import torch

from tests.test_abi_host import FAKE, INVALID, UNSUPPORTED, Pool, decode, good_pool, lib  # noqa: F401

pk = pytest.importorskip("paged_kv_flash_gb300.pagedkv")
V = ctypes.c_void_p


def int4_pool(**kw):
    return good_pool(**{"dtype": 4, **kw})


@pytest.mark.parametrize("bad", [dict(head_dim=64), dict(page_size=32), dict(num_kv_heads=0),
                                 dict(k=None), dict(v=FAKE + 8), dict(k_scale=FAKE),
                                 dict(v_scale=FAKE), dict(dtype=3), dict(dtype=2)])
def test_append_and_decode_refuse_bad_pools(lib, bad):  # noqa: F811
    f = lib.pkv_kv_append
    f.restype = ctypes.c_int32
    args = [V(FAKE), V(FAKE), 0, V(FAKE), 1, V(FAKE), 4, V(FAKE), None, None]
    assert f(ctypes.byref(int4_pool(**bad)), *args) == INVALID
    assert f(ctypes.byref(int4_pool()), *args) == 0              # no tokens: nothing launched
    assert decode(lib, int4_pool(**bad)) == INVALID


def unpack(lib, src, dst, **kw):  # noqa: F811
    a = dict(B=1, st=FAKE, sp=4, dt=FAKE, dp=4, starts=None, lens=FAKE, L=64, w=None)
    a.update(kw)
    f = lib.pkv_kv_unpack
    f.restype = ctypes.c_int32
    return f(ctypes.byref(src), ctypes.byref(dst), a["B"], V(a["st"]), a["sp"], V(a["dt"]), a["dp"],
             V(a["starts"]), V(a["lens"]), a["L"], V(a["w"]), None)


@pytest.mark.parametrize("bad", [dict(B=-1), dict(sp=0), dict(dp=3), dict(L=65), dict(L=-1),
                                 dict(st=None), dict(dt=None), dict(lens=None), dict(w=FAKE + 4)])
def test_unpack_refuses_bad_arguments(lib, bad):  # noqa: F811
    assert unpack(lib, int4_pool(), good_pool(), **bad) == INVALID


def test_unpack_refuses_bad_pools(lib):  # noqa: F811
    assert unpack(lib, good_pool(), good_pool()) == UNSUPPORTED          # bf16 source
    assert unpack(lib, int4_pool(), int4_pool()) == INVALID              # destination not bf16
    assert unpack(lib, int4_pool(), good_pool(num_kv_heads=4)) == INVALID
    assert unpack(lib, int4_pool(num_kv_heads=1 << 30), good_pool(num_kv_heads=1 << 30)) == UNSUPPORTED
    assert unpack(lib, int4_pool(), good_pool(), B=65536) == UNSUPPORTED
    assert unpack(lib, int4_pool(), good_pool(), B=0) == 0
    assert unpack(lib, int4_pool(), good_pool(), L=0) == 0


def test_prefill_and_fused_inputs_take_no_4bit_pool(lib):  # noqa: F811
    f = lib.pkv_paged_attn_prefill
    f.restype = ctypes.c_int32
    args = [V(FAKE), 16, V(FAKE), 1, 4, V(FAKE), 4, V(FAKE), 16, ctypes.c_float(0.1), V(FAKE),
            ctypes.c_size_t(1 << 30), 0, V(FAKE), None, None]
    assert f(ctypes.byref(int4_pool()), *args) == UNSUPPORTED


def test_binding_checks_4bit_pools(monkeypatch):
    def need(t, dtype, name):
        if t.dtype != dtype or not t.is_contiguous():
            raise ValueError(f"{name}: expected a contiguous {dtype} tensor")
    pool = pk.Pool.empty(4, 2, dtype=torch.uint8, device="cpu")
    with pytest.raises(ValueError, match="pool.k"):
        pool.c()                                               # host memory
    monkeypatch.setattr(pk, "_need", need)
    u8 = lambda *s: torch.zeros(s, dtype=torch.uint8)  # noqa: E731
    pk.Pool(u8(4, 2, 1152), u8(4, 2, 1152))._validate()
    c = pk.Pool(u8(4, 2, 1152), u8(4, 2, 1152)).c()
    assert (c.num_pages, c.num_kv_heads, c.page_size, c.head_dim, c.dtype) == (4, 2, 16, 128, 4)
    f32 = torch.zeros(4, 2, 16)
    for bad in (pk.Pool(u8(4, 2, 1024), u8(4, 2, 1024)), pk.Pool(u8(4, 2, 16, 72), u8(4, 2, 16, 72)),
                pk.Pool(u8(4, 2, 1152), u8(5, 2, 1152)),
                pk.Pool(u8(4, 2, 1152), torch.zeros((4, 2, 16, 128), dtype=torch.int8)),
                pk.Pool(u8(4, 2, 1152), u8(4, 2, 1152), f32, f32)):
        with pytest.raises(ValueError):
            bad._validate()


def test_binding_refuses_tensors_of_another_device(monkeypatch):
    """Every tensor of a call lies on one device, the current one (the checks
    alone, on stand-ins for CUDA tensors)."""
    monkeypatch.setattr(torch.cuda, "current_device", lambda: 0)

    class T:
        is_cuda, dtype = True, torch.int32

        def __init__(self, i):
            self.device = torch.device("cuda", i)

        def get_device(self):
            return self.device.index

        def is_contiguous(self):
            return True

    pk._need(T(1), torch.int32, "x", 1)
    pk._on(0, T(0), None, T(0))
    with pytest.raises(ValueError, match="cuda:1"):
        pk._need(T(1), torch.int32, "x", 0)
    with pytest.raises(ValueError, match="cuda:1"):
        pk._on(0, T(0), T(1))
    with pytest.raises(ValueError, match="current device"):
        pk._stream(None, 1)


def test_unpack_binding_refuses_mismatched_tables(monkeypatch):
    monkeypatch.setattr(pk, "_need", lambda *a: None)
    src, dst = pk.Pool.empty(4, 2, dtype=torch.uint8, device="cpu"), pk.Pool.empty(4, 2, device="cpu")
    bt, lens = torch.zeros((2, 4), dtype=torch.int32), torch.zeros(2, dtype=torch.int32)
    for kw in (dict(a=bt[:1]), dict(b=bt[:1]), dict(starts=lens[:1]), dict(k_smooth=torch.ones(64))):
        a, b = kw.pop("a", bt), kw.pop("b", bt)
        with pytest.raises(ValueError):
            pk.kv_unpack(src, dst, a, b, lens, 64, **kw)


# --------------------------------------------------------------- page tables

def tables(lib, **kw):  # noqa: F811
    a = dict(lens=FAKE, new=FAKE, B=4, ring=FAKE, cap=64, state=FAKE, pages=64, bt=FAKE, mp=8,
             out=FAKE, cu=FAKE, offs=FAKE, slots=FAKE, sc=4, so=FAKE)
    a.update(kw)
    f = lib.pkv_page_tables
    f.restype = ctypes.c_int32
    return f(V(a["lens"]), V(a["new"]), a["B"], V(a["ring"]), a["cap"], V(a["state"]), a["pages"],
             V(a["bt"]), a["mp"], V(a["out"]), V(a["cu"]), V(a["offs"]), V(a["slots"]), a["sc"],
             V(a["so"]), None)


@pytest.mark.parametrize("bad", [dict(B=-1), dict(cap=0), dict(pages=0), dict(mp=0), dict(sc=-1),
                                 dict(slots=None)] +
                         [{n: None} for n in ("lens", "new", "ring", "state", "bt", "out", "cu",
                                              "offs", "so")])
def test_page_tables_refuses_bad_arguments(lib, bad):  # noqa: F811
    assert tables(lib, **bad) == INVALID


def test_page_tables_limits(lib):  # noqa: F811
    assert tables(lib, B=0) == 0
    assert tables(lib, pages=1 << 27) == UNSUPPORTED            # slots pass 31 bits
    assert tables(lib, mp=1 << 27) == UNSUPPORTED
    assert tables(lib, B=2147483647) == UNSUPPORTED


def test_page_tables_refuses_arrays_that_overlap(lib):  # noqa: F811
    """Each array a page apart, then each pair of them on one another; the two
    states may be their own inputs, but not overlap them in part."""
    names = ["lens", "new", "ring", "state", "bt", "out", "cu", "offs", "slots", "so"]
    apart = {n: FAKE + 4096 * i for i, n in enumerate(names)}
    for i, a in enumerate(names):
        for b in names[i + 1:]:
            if (a, b) in (("lens", "out"), ("state", "so")):
                assert tables(lib, **{**apart, b: apart[a] + 4}) == INVALID
            else:
                assert tables(lib, **{**apart, b: apart[a]}) == INVALID
    assert tables(lib, **{**apart, "cu": apart["bt"] + 4 * 31}) == INVALID       # its last entry


def test_page_tables_binding_checks_sizes(monkeypatch):
    monkeypatch.setattr(pk, "_need", lambda *a: None)
    i = lambda *s: torch.zeros(s, dtype=torch.int32)  # noqa: E731
    good = dict(seq_lens=i(3), new_lens=i(3), block_table=i(3, 4), free_ring=i(9), ring_state=i(2),
                num_pages=9)
    for bad in (dict(new_lens=i(2)), dict(block_table=i(2, 4)), dict(block_table=i(12)),
                dict(ring_state=i(3)), dict(cu_new=i(3)), dict(page_offsets=i(2, 3)),
                dict(seq_lens_out=i(4)), dict(ring_state_out=i(1))):
        with pytest.raises(ValueError):
            pk.page_tables(**{**good, **bad})


# ------------------------------------------------------------------- attention

@pytest.mark.parametrize("bad", [dict(Hq=3), dict(q=None), dict(out=None), dict(B=-1),
                                 dict(max_seq_len=65), dict(scale=float("nan")), dict(splits=-2),
                                 dict(q=FAKE + 8), dict(smooth=FAKE + 4)])
def test_int4_decode_refuses_bad_arguments(lib, bad):  # noqa: F811
    assert decode(lib, int4_pool(), **bad) == INVALID


def test_int4_decode_takes_any_group_and_checks_its_workspace(lib):  # noqa: F811
    assert decode(lib, int4_pool(), B=0, Hq=6) == 0
    assert decode(lib, int4_pool(), Hq=6, splits=4) == INVALID           # no workspace
    assert decode(lib, int4_pool(num_kv_heads=65536), Hq=65536) == UNSUPPORTED
    s, c, w, z = ctypes.c_int32(), ctypes.c_int32(), ctypes.c_size_t(), ctypes.c_size_t()
    assert lib.pkv_decode_plan(1, 12, 2, 64, 4, 4, ctypes.byref(s), ctypes.byref(c),
                               ctypes.byref(w), ctypes.byref(z)) == 0
    assert (s.value, c.value, z.value) == (4, 1, 65536 * 4)
    assert decode(lib, int4_pool(), Hq=12, splits=4, ws=FAKE, ws_bytes=w.value - 1) == INVALID


def multi(lib, name, pool, **kw):  # noqa: F811
    a = dict(q=FAKE, T=4, cu=FAKE, B=2, Hq=4, bt=FAKE, mp=4, sl=FAKE, mq=2, L=64, scale=0.1,
             smooth=None, splits=1, ws=None, wsb=0, out=FAKE)
    a.update(kw)
    f = getattr(lib, name)
    f.restype = ctypes.c_int32
    smooth = [V(a["smooth"])] if name.endswith("int4") else []
    return f(ctypes.byref(pool), V(a["q"]), a["T"], V(a["cu"]), a["B"], a["Hq"], V(a["bt"]), a["mp"],
             V(a["sl"]), a["mq"], a["L"], ctypes.c_float(a["scale"]), *smooth, a["splits"],
             V(a["ws"]), ctypes.c_size_t(a["wsb"]), V(a["out"]), None, None)


@pytest.mark.parametrize("bad", [dict(Hq=3), dict(q=FAKE + 4), dict(out=FAKE + 4), dict(mq=0),
                                 dict(L=65), dict(splits=2), dict(smooth=FAKE + 8), dict(cu=None),
                                 dict(scale=float("inf"))])
def test_int4_verify_refuses_bad_arguments(lib, bad):  # noqa: F811
    assert multi(lib, "pkv_paged_attn_decode_multi_int4", int4_pool(), **bad) == INVALID


def test_int4_verify_is_for_4bit_pools(lib):  # noqa: F811
    name = "pkv_paged_attn_decode_multi_int4"
    assert multi(lib, name, good_pool()) == UNSUPPORTED
    assert multi(lib, "pkv_paged_attn_decode_multi", int4_pool()) == UNSUPPORTED
    assert multi(lib, name, int4_pool(), mq=17) == UNSUPPORTED
    assert multi(lib, name, int4_pool(num_kv_heads=40000), Hq=80000 * 16, mq=16) == UNSUPPORTED
    assert multi(lib, name, int4_pool(), T=0) == 0


def test_verify_binding_refuses_weights_for_bf16_pools(monkeypatch):
    monkeypatch.setattr(pk, "_need", lambda *a: None)
    monkeypatch.setattr(pk, "_stream", lambda *a: None)
    q = torch.zeros((1, 4, 128), dtype=torch.bfloat16)
    i = torch.zeros(2, dtype=torch.int32)
    ws = torch.zeros(256, dtype=torch.uint8)
    pool = pk.Pool.empty(4, 2, device="cpu")
    with pytest.raises(ValueError, match="k_smooth"):
        pk.paged_attn_decode_multi(pool, q, i, i.view(1, 2), i[:1], 1, 16, 0.1, workspace=ws,
                                   k_smooth=torch.ones(128))
