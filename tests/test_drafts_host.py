"""Host-side checks of the operators that check drafted tokens (no GPU needed,
no kernel launched): the C ABI's refusals and the binding's checks."""
import ctypes
import os

import pytest

import mxfp4_microscaling_quantization_mxq_amd as mxq

torch = pytest.importorskip("torch")

INVALID, MISALIGNED, NOT_SUPPORTED = 1, 2, 3
# Fake device addresses: every call below fails validation before anything is enqueued.
A, B, C, D, E, F, G = (ctypes.c_void_p(0x1000000 * (i + 1)) for i in range(7))
MIS, MIS2, MIS4 = ctypes.c_void_p(0x1000008), ctypes.c_void_p(0x1000002), ctypes.c_void_p(0x1000004)
NULL = ctypes.c_void_p(0)


@pytest.fixture(scope="module")
def lib():
    if not os.path.exists(mxq.LIB_PATH):
        pytest.skip("libmxq.so not built")
    return mxq.capi()


def rope(lib, q=A, qs=512, k=B, ks=256, v=C, vs=256, dt=1, pos=D, axes=1, axis=NULL, freqs=E, pairs=64, inter=0,
         slots=F, tokens=3, qh=4, pages=9, heads=2, page=16, dim=128, fmt=0, kq=A, ksc=B, vq=C, vsc=D, out=G):
    return lib.mxq_rope_append(q, qs, k, ks, v, vs, dt, pos, axes, axis, freqs, pairs, inter, slots, tokens, qh, pages,
                               heads, page, dim, fmt, kq, ksc, vq, vsc, out, NULL)


def test_rope_refusals(lib):
    for bad in (dict(q=NULL), dict(k=NULL), dict(v=NULL), dict(pos=NULL), dict(freqs=NULL), dict(slots=NULL),
                dict(out=NULL), dict(kq=NULL), dict(vsc=NULL), dict(dt=2), dict(fmt=2), dict(qs=504), dict(ks=248),
                dict(vs=252), dict(qs=516), dict(tokens=0), dict(tokens=-1), dict(tokens=(1 << 22) + 1),
                dict(qh=0), dict(qh=-4), dict(heads=0), dict(page=8), dict(page=24), dict(dim=48), dict(pages=0),
                dict(dim=544, qs=4096, ks=4096, vs=4096), dict(pairs=0), dict(pairs=4), dict(pairs=12), dict(pairs=72),
                dict(pairs=-8), dict(axes=0), dict(axes=257, axis=A), dict(axes=3), dict(axes=1, axis=A),
                dict(qh=1 << 14, qs=1 << 21), dict(qs=1 << 60),
                # the output over an input
                dict(out=A), dict(out=B), dict(out=C), dict(out=ctypes.c_void_p(0x1000000 + 16)),
                dict(out=ctypes.c_void_p(0x1000000 - 16))):
        assert rope(lib, **bad) == INVALID, bad
    for bad in (dict(q=MIS), dict(k=MIS), dict(v=MIS), dict(out=ctypes.c_void_p(0x9000008)), dict(kq=MIS),
                dict(vsc=MIS), dict(pos=MIS4), dict(slots=MIS4), dict(freqs=MIS2)):
        assert rope(lib, **bad) == MISALIGNED, bad


def test_no_device_reports_not_supported(lib):
    if torch.cuda.device_count() > 0:
        pytest.skip("a GPU is present: this case is only safe without one")
    assert rope(lib) == NOT_SUPPORTED
    assert rope(lib, axes=3, axis=A, inter=1) == NOT_SUPPORTED


# ------------------------------------------------------------------ the binding's checks, on host tensors

def test_binding_rope():
    c = mxq.kv_cache(3, 16, 2, 64, device="cpu")
    q, k = torch.zeros(5, 4, 64), torch.zeros(5, 2, 64)
    n, p, f = torch.zeros(5, dtype=torch.int64), torch.zeros(5, dtype=torch.int64), torch.ones(32)
    p3, a3 = torch.zeros(3, 5, dtype=torch.int64), torch.zeros(32, dtype=torch.uint8)
    for args, kw in (((q, k[:4], k, n, p, f), {}), ((q[:4], k, k, n, p, f), {}), ((q, k, k[:, :1], n, p, f), {}),
                     ((q[..., :32], k, k, n, p, f), {}), ((q, k, k, n[:4], p, f), {}), ((q, k, k, n, p[:4], f), {}),
                     ((q, k, k, n, p3, f), {}), ((q, k, k, n, p, f), dict(axes=a3)), ((q, k, k, n, p3[:1], f), dict(axes=a3)),
                     ((q, k, k, n, p3, f), dict(axes=a3[:16])), ((q, k, k, n, p, f[None]), {}),
                     ((q, k, k, n, p3[:, :4], f), dict(axes=a3)),
                     ((q, k, k, n, p, f), dict(out=torch.zeros(5, 2, 64, dtype=torch.bfloat16))),
                     ((q.transpose(0, 1), k, k, n, p, f), {}), ((q, k, k, n, p, f), {})):  # the last: host tensors
        with pytest.raises(ValueError):
            mxq.rope_append(c, *args, **kw)
    for args, kw in (((q.half(), k.half(), k.half(), n, p, f), {}), ((q, k.bfloat16(), k, n, p, f), {}),
                     ((q, k, k.bfloat16(), n, p, f), {}), ((q, k, k, n.int(), p, f), {}), ((q, k, k, n, p.int(), f), {}),
                     ((q, k, k, n, p, f.double()), {}), ((q, k, k, n, p3, f), dict(axes=a3.int())),
                     ((q, k, k, n, p, f), dict(out=torch.zeros(5, 4, 64)))):
        with pytest.raises(TypeError):
            mxq.rope_append(c, *args, **kw)
