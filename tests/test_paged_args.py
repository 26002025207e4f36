"""Host argument checks of the paged 4-bit cache (include/tq.h), without a
device: every refusal comes before anything is enqueued.  The checks that need
a handle get one laid out like the library's own {head_dim, page_size, device,
status}, with a device number that no machine has, so a call that passes every
check ends in TQ_ERR_DEVICE (or TQ_ERR_CUDA without a driver)."""
import ctypes

import pytest

tq = pytest.importorskip("kv_cache_vector_10_b200")
lib = tq.lib


class Handle(ctypes.Structure):
    _fields_ = [("d", ctypes.c_int), ("page", ctypes.c_int), ("device", ctypes.c_int), ("status", ctypes.c_void_p)]


P = 1 << 20          # an aligned address that is never dereferenced


def handle(d=128, page=64):
    return Handle(d, page, 9999, None)


def name(code):
    return tq.STATUS_NAMES[code]


PASSED = ("TQ_ERR_DEVICE", "TQ_ERR_CUDA")


def test_create_refuses():
    out = ctypes.c_void_p()
    assert name(lib.tq_paged_create(128, 64, None)) == "TQ_ERR_NULL"
    for d, page, want in [(0, 64, "TQ_ERR_ZERO_DIM"), (96, 64, "TQ_ERR_DIM"), (512, 64, "TQ_ERR_DIM"),
                          (128, 0, "TQ_ERR_DIM_MISMATCH"), (128, 8, "TQ_ERR_DIM_MISMATCH"),
                          (128, 48, "TQ_ERR_DIM_MISMATCH"), (128, 512, "TQ_ERR_DIM_MISMATCH")]:
        assert name(lib.tq_paged_create(d, page, ctypes.byref(out))) == want
        assert out.value is None
    lib.tq_paged_destroy(None)
    assert lib.tq_paged_page_bytes(None) == 0
    for d, page in [(64, 16), (128, 64), (256, 256)]:
        h = handle(d, page)
        assert lib.tq_paged_page_bytes(ctypes.byref(h)) == page * (d // 2 + d // 32)


def _write(h, pages, k=P, v=P, dtype=1, n=4, sk=(256, 128), sv=(256, 128), slots=P, ks=None, vs=None):
    return name(lib.tq_paged_write(ctypes.byref(h), k, v, dtype, n, *sk, *sv, slots, ctypes.byref(pages), ks, vs, None))


def test_write_refuses():
    h, pages = handle(), tq.tq_pages(P, P, 10, 2, 0)
    assert _write(h, pages) in PASSED
    assert _write(h, pages, n=0, k=None, v=None, slots=None) in PASSED + ("TQ_OK",)
    assert name(lib.tq_paged_write(None, P, P, 1, 4, 0, 0, 0, 0, P, ctypes.byref(pages), None, None, None)) == "TQ_ERR_NULL"
    assert name(lib.tq_paged_write(ctypes.byref(h), P, P, 1, 4, 0, 0, 0, 0, P, None, None, None, None)) == "TQ_ERR_NULL"
    assert _write(h, pages, k=None, v=None) == "TQ_ERR_NULL"
    assert _write(h, pages, k=None, ks=P) == "TQ_ERR_NULL"
    assert _write(h, tq.tq_pages(None, P, 10, 2, 0)) == "TQ_ERR_NULL"
    assert _write(h, tq.tq_pages(P, P, 0, 2, 0)) == "TQ_ERR_EMPTY"
    assert _write(h, tq.tq_pages(P, P, 10, 0, 0)) == "TQ_ERR_EMPTY"
    assert _write(h, tq.tq_pages(P, P, 10, 2000, 0)) == "TQ_ERR_LIMIT"
    assert _write(h, tq.tq_pages(P + 8, P, 10, 2, 0)) == "TQ_ERR_ALIGN"
    assert _write(h, pages, dtype=7) == "TQ_ERR_DIM_MISMATCH"
    assert _write(h, pages, n=-1) == "TQ_ERR_DIM_MISMATCH"
    for bad in [dict(k=P + 2), dict(v=P + 8), dict(ks=P + 16), dict(sk=(257, 128)), dict(sv=(256, 4))]:
        assert _write(h, pages, **bad) == "TQ_ERR_ALIGN", bad
    assert _write(h, pages, dtype=0, sk=(260, 4)) in PASSED      # float32: multiples of four elements


def test_read_refuses():
    h, pages = handle(), tq.tq_pages(P, P, 10, 2, 0)

    def read(ko=P, vo=P, n=4, dtype=2, pages=pages):
        return name(lib.tq_paged_read(ctypes.byref(h), ctypes.byref(pages), P, n, ko, vo, dtype, None))

    assert read() in PASSED and read(ko=None) in PASSED
    assert read(ko=None, vo=None) == "TQ_ERR_NULL"
    assert read(dtype=3) == "TQ_ERR_DIM_MISMATCH" and read(n=-2) == "TQ_ERR_DIM_MISMATCH"
    assert read(vo=P + 16) == "TQ_ERR_ALIGN"
    assert read(n=1 << 31) in PASSED + ("TQ_ERR_LIMIT",)
    assert read(pages=tq.tq_pages(P, None, 10, 2, 0)) == "TQ_ERR_NULL"


def _attend(h, **kw):
    a = dict(pages=tq.tq_pages(P, P, 10, 2, 0), q=P, dtype=1, total=3, heads=8, sq=(1024, 128), table=P, stride=5, pages_max=5,
             lens=P, starts=P, batch=2, most=2, window=0, sinks=0, scale=0.0, out=P, so=(1024, 128), ws=P, ws_bytes=1 << 40)
    a.update(kw)
    return name(lib.tq_paged_attention(ctypes.byref(h), ctypes.byref(a["pages"]), a["q"], a["dtype"], a["total"], a["heads"],
                                       *a["sq"], a["table"], a["stride"], a["pages_max"], a["lens"], a["starts"], a["batch"],
                                       a["most"], a["window"], a["sinks"], a["scale"], a["out"], *a["so"], a["ws"],
                                       a["ws_bytes"], None))


def test_attention_refuses():
    h = handle()
    assert _attend(h) in PASSED
    for bad in [dict(q=None), dict(out=None), dict(lens=None), dict(table=None), dict(pages=tq.tq_pages(P, None, 10, 2, 0))]:
        assert _attend(h, **bad) == "TQ_ERR_NULL", bad
    for bad in [dict(batch=0), dict(heads=0), dict(most=0)]:
        assert _attend(h, **bad) == "TQ_ERR_EMPTY", bad
    for bad in [dict(dtype=0), dict(dtype=5), dict(heads=7), dict(total=-1), dict(starts=None), dict(stride=4), dict(window=-1),
                dict(sinks=-1), dict(scale=-1.0), dict(scale=float("nan")), dict(pages_max=-1, stride=0)]:
        assert _attend(h, **bad) == "TQ_ERR_DIM_MISMATCH", bad
    for bad in [dict(heads=2048), dict(batch=70000), dict(total=1 << 28), dict(total=1 << 62),
                dict(pages_max=1 << 25, stride=1 << 25), dict(pages_max=1 << 60, stride=1 << 60), dict(window=1 << 30)]:
        assert _attend(h, **bad) == "TQ_ERR_LIMIT", bad
    for bad in [dict(q=P + 8), dict(out=P + 4), dict(sq=(1028, 128)), dict(so=(1024, 4)), dict(lens=P + 2), dict(starts=P + 1),
                dict(table=P + 2)]:
        assert _attend(h, **bad) == "TQ_ERR_ALIGN", bad


def test_workspace_bytes():
    h = handle()
    ws = lambda *a: lib.tq_paged_workspace_bytes(ctypes.byref(h), *a)   # noqa: E731
    assert lib.tq_paged_workspace_bytes(None, 8, 2, 1, 4, 1) == 0
    for bad in [(0, 2, 1, 4, 1), (8, 0, 1, 4, 1), (7, 2, 1, 4, 1), (8, 2, 0, 4, 1), (8, 2, 1, -1, 1), (8, 2, 1, 4, 0),
                (8, 2, 1, 1 << 25, 1), (8, 2, 1, 1 << 60, 1)]:
        assert ws(*bad) == 0, bad
    assert ws(8, 2, 1, 4, 1) == 0 and ws(8, 2, 1, 2, 40) == 0       # short sequences are not split
    assert 0 < ws(8, 2, 1, 40, 1) <= ws(8, 2, 64, 40, 1) <= ws(8, 2, 64, 4000, 1)
    assert 0 < ws(8, 2, 1, 40, 40) <= ws(8, 2, 64, 40, 40)
    assert ws(1024, 1024, 65535, 1 << 20, 1) < 1 << 26          # bounded by the GPU's size, not by the batch


def test_status_calls_refuse_null():
    assert name(lib.tq_paged_get_status(None, None, None, None)) == "TQ_ERR_NULL"
    assert name(lib.tq_paged_reset_status(None, None)) == "TQ_ERR_NULL"
