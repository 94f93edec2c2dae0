"""Host-side checks of the serving operators (no GPU needed, no kernel
launched): the C ABI's refusals, the workspace sizes and the binding's checks."""
import ctypes
import os

import pytest

import mxfp4_microscaling_quantization_mxq_amd as mxq

torch = pytest.importorskip("torch")

INVALID, MISALIGNED, NOT_SUPPORTED = 1, 2, 3
# Fake device addresses: every call below fails validation before anything is enqueued.
A, B, C, D, E = (ctypes.c_void_p(0x10000 * (i + 1)) for i in range(5))
MIS, MIS2 = ctypes.c_void_p(0x10008), ctypes.c_void_p(0x10002)
NULL = ctypes.c_void_p(0)


@pytest.fixture(scope="module")
def lib():
    if not os.path.exists(mxq.LIB_PATH):
        pytest.skip("libmxq.so not built")
    return mxq.capi()


def test_norm_refusals(lib):
    def call(x=A, res=B, w=C, dt=1, rows=4, k=64, eps=1e-6, r=D, q=E, s=A):
        return lib.mxq_rmsnorm_quantize_fp8(x, res, w, dt, rows, k, eps, r, q, s, NULL)

    for bad in (dict(k=48), dict(k=0), dict(rows=0), dict(rows=-1), dict(dt=2), dict(x=NULL), dict(w=NULL),
                dict(q=NULL), dict(s=NULL), dict(r=NULL), dict(eps=0.0), dict(eps=-1.0), dict(eps=float("nan")),
                dict(eps=float("inf")), dict(rows=2 ** 62)):
        assert call(**bad) == INVALID, bad
    for bad in (dict(x=MIS), dict(res=MIS), dict(w=MIS), dict(r=MIS), dict(q=MIS), dict(s=MIS)):
        assert call(**bad) == MISALIGNED, bad


def test_cache_refusals(lib):
    def append(k=A, ks=256, v=B, vs=256, dt=1, slots=C, tokens=3, pages=9, heads=2, page=16, dim=128, fmt=0, kq=A,
               ksc=B, vq=C, vsc=D):
        return lib.mxq_kv_append(k, ks, v, vs, dt, slots, tokens, pages, heads, page, dim, fmt, kq, ksc, vq, vsc, NULL)

    def read(kq=A, ksc=B, vq=C, vsc=D, slots=E, tokens=3, pages=9, heads=2, page=16, dim=128, fmt=0, k=A, v=B, dt=1):
        return lib.mxq_kv_read(kq, ksc, vq, vsc, slots, tokens, pages, heads, page, dim, fmt, k, v, dt, NULL)

    shape = (dict(pages=0), dict(heads=0), dict(page=8), dict(page=24), dict(page=2048), dict(dim=48), dict(dim=0),
             dict(dim=-32), dict(heads=1 << 20), dict(pages=2 ** 61), dict(fmt=2), dict(fmt=-1), dict(dt=3),
             dict(tokens=0), dict(tokens=-1), dict(k=NULL), dict(v=NULL), dict(slots=NULL), dict(kq=NULL),
             dict(ksc=NULL), dict(vq=NULL), dict(vsc=NULL))
    for bad in shape + (dict(ks=248), dict(vs=255), dict(ks=260), dict(tokens=2 ** 60)):
        assert append(**bad) == INVALID, bad
    for bad in shape:
        assert read(**bad) == INVALID, bad
    for name in ("k", "v", "kq", "ksc", "vq", "vsc"):
        assert append(**{name: MIS}) == MISALIGNED and read(**{name: MIS}) == MISALIGNED, name
    assert append(slots=MIS2) == MISALIGNED and read(slots=MIS2) == MISALIGNED


def attend(lib, q=A, qs=1024, kq=A, ks=B, vq=C, vs=D, table=E, width=4, stride=4, lens=A, sinks=NULL, batch=2, qh=8,
           pages=9, heads=2, page=16, dim=128, fmt=0, scale=0.1, window=0, ws=A, ws_bytes=1 << 30, out=B, dt=1):
    return lib.mxq_paged_attention(q, qs, kq, ks, vq, vs, table, width, stride, lens, sinks, batch, qh, pages, heads,
                                   page, dim, fmt, scale, window, ws, ws_bytes, out, dt, NULL)


def test_attention_refusals(lib):
    for bad in (dict(q=NULL), dict(table=NULL), dict(lens=NULL), dict(out=NULL), dict(kq=NULL), dict(vs=NULL),
                dict(batch=0), dict(qh=7), dict(qh=0), dict(heads=3), dict(dim=96), dict(dim=32), dict(dim=512),
                dict(page=20), dict(width=0), dict(stride=3), dict(qs=1016), dict(qs=1028), dict(window=-1),
                dict(scale=float("nan")), dict(scale=float("inf")), dict(dt=2), dict(fmt=2), dict(batch=2 ** 40),
                dict(width=2 ** 31, stride=2 ** 31), dict(batch=1 << 24)):
        assert attend(lib, **bad) == INVALID, bad
    for bad in (dict(q=MIS), dict(out=MIS), dict(kq=MIS), dict(vs=MIS), dict(table=MIS2), dict(lens=MIS2),
                dict(sinks=MIS2)):
        assert attend(lib, **bad) == MISALIGNED, bad


def workspace(lib, batch, qh, heads, page, dim, width, window=0):
    n = ctypes.c_int64(-1)
    code = lib.mxq_paged_attention_workspace(batch, qh, heads, page, dim, width, window, ctypes.byref(n))
    return code, n.value


def test_attention_workspace(lib):
    code, need = workspace(lib, 1, 8, 2, 16, 128, 4096)
    assert code == 0 and need > 0 and need % 4 == 0
    big = dict(batch=1, width=4096, stride=4096, qs=1024)
    assert attend(lib, ws_bytes=need - 1, **big) == INVALID
    assert attend(lib, ws=NULL, ws_bytes=need, **big) == INVALID
    assert attend(lib, ws=MIS, ws_bytes=need, **big) == MISALIGNED
    # a short table leaves nothing to split
    assert workspace(lib, 1, 8, 2, 16, 128, 1) == (0, 0)
    # a window bounds what is split
    assert workspace(lib, 1, 8, 2, 16, 128, 4096, 64)[1] < need
    assert workspace(lib, 1, 8, 3, 16, 128, 4096)[0] == INVALID
    assert workspace(lib, 1, 8, 2, 16, 96, 4096)[0] == INVALID
    assert lib.mxq_paged_attention_workspace(1, 8, 2, 16, 128, 4, 0, None) == INVALID


def test_no_device_reports_not_supported(lib):
    if torch.cuda.device_count() > 0:
        pytest.skip("a GPU is present: this case is only safe without one")
    assert lib.mxq_rmsnorm_quantize_fp8(A, B, C, 1, 4, 64, 1e-6, D, E, A, NULL) == NOT_SUPPORTED
    assert attend(lib) == NOT_SUPPORTED


# ------------------------------------------------------------------ the binding's checks, on host tensors

def cpu_cache(fmt="mxfp8"):
    return mxq.kv_cache(3, 16, 2, 64, fmt, device="cpu")


def test_kv_cache_shapes():
    for fmt, w in (("mxfp8", 64), ("mxfp4", 32)):
        c = cpu_cache(fmt)
        assert [tuple(t.shape) for t in c] == [(3, 2, 16, w), (3, 2, 16, 2), (3, 2, 16, w), (3, 2, 2, 16)]
    with pytest.raises(ValueError):
        mxq.kv_cache(3, 16, 2, 64, "fp16", device="cpu")
    with pytest.raises(ValueError):
        mxq.kv_cache(3, 16, 2, 72, device="cpu")


def test_binding_norm():
    x, w = torch.zeros(4, 64), torch.ones(64)
    for args, kw in (((x[:, :48], w[:48]), {}), ((x, w[:32]), {}), ((x[:, ::2], w), {}),
                     ((x, w), dict(residual=x[:2])), ((x, w), dict(eps=0.0)), ((x, w), dict(r=torch.zeros(4, 64))),
                     ((x, w), {})):  # the last: host tensors
        with pytest.raises(ValueError):
            mxq.rmsnorm_quantize_fp8(*args, **kw)
    for args, kw in (((x.half(), w), {}), ((x, w.bfloat16()), {}), ((x, w), dict(residual=x.bfloat16())),
                     ((x, w), dict(q=torch.zeros(4, 64)))):
        with pytest.raises(TypeError):
            mxq.rmsnorm_quantize_fp8(*args, **kw)


def test_binding_cache():
    c = cpu_cache()
    k, slots = torch.zeros(5, 2, 64), torch.zeros(5, dtype=torch.int64)
    for cache, a, b, sl in ((c, k[:, :1], k, slots), (c, k, k[:4], slots), (c, k, k, slots[:4]),
                            (c, k[..., :32], k, slots), (c, k.transpose(0, 1), k, slots),
                            (c, torch.zeros(5, 2, 128)[..., ::2], k, slots), (c, k, k, slots),
                            (c._replace(vs=c.ks), k, k, slots), (c._replace(kq=c.kq[..., :48]), k, k, slots),
                            (c._replace(ks=c.ks[..., :1].contiguous()), k, k, slots)):
        with pytest.raises(ValueError):
            mxq.kv_append(cache, a, b, sl)
    for a, b, sl in ((k.half(), k.half(), slots), (k, k.bfloat16(), slots), (k, k, slots.int())):
        with pytest.raises(TypeError):
            mxq.kv_append(c, a, b, sl)
    with pytest.raises(ValueError):
        mxq.kv_read(c, slots)  # host tensors
    with pytest.raises(TypeError):
        mxq.kv_read(c, slots, dtype=torch.float16)


def test_binding_attention():
    c = cpu_cache()
    q, table, lens = torch.zeros(2, 4, 64, dtype=torch.bfloat16), torch.zeros(2, 3, dtype=torch.int32), torch.zeros(
        2, dtype=torch.int32)
    for a, t, n, kw in ((q[:, :3], table, lens, {}), (q, table[:1], lens, {}), (q, table, lens[:1], {}),
                        (q, table.t().contiguous().t(), lens, {}), (q[..., :32], table, lens, {}),
                        (q, table, lens, dict(sinks=torch.zeros(3))), (q, table, lens, {}),
                        (q, table, lens, dict(out=torch.zeros(2, 4, 32, dtype=torch.bfloat16)))):
        with pytest.raises(ValueError):
            mxq.paged_attention(a, c, t, n, **kw)
    for a, t, n, kw in ((q.float(), table, lens, {}), (q, table.long(), lens, {}), (q, table, lens.long(), {}),
                        (q, table, lens, dict(out_dtype=torch.float16)),
                        (q, table, lens, dict(sinks=torch.zeros(4, dtype=torch.bfloat16)))):
        with pytest.raises(TypeError):
            mxq.paged_attention(a, c, t, n, **kw)
    with pytest.raises(mxq.MXQError):
        mxq.paged_attention(q, c, table, lens, window=-1)
