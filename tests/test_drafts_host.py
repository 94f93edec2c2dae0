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


# ------------------------------------------------------------------ attention of a tree

def tree(lib, q=A, qs=1024, kq=A, ks=B, vq=C, vs=D, table=E, width=4, stride=4, context=A, mask=B, sinks=NULL, batch=2,
         drafts=5, qh=8, pages=9, heads=2, page=16, dim=128, fmt=0, scale=0.1, window=0, first=0, ws=A,
         ws_bytes=1 << 30, out=B, dt=1):
    return lib.mxq_tree_attention(q, qs, kq, ks, vq, vs, table, width, stride, context, mask, sinks, batch, drafts, qh,
                                  pages, heads, page, dim, fmt, scale, window, first, ws, ws_bytes, out, dt, NULL)


def test_tree_refusals(lib):
    for bad in (dict(q=NULL), dict(table=NULL), dict(context=NULL), dict(mask=NULL), dict(out=NULL), dict(kq=NULL),
                dict(vs=NULL), dict(batch=0), dict(drafts=0), dict(drafts=-1), dict(drafts=257), dict(qh=7), dict(qh=0),
                dict(heads=3), dict(dim=96), dict(dim=32), dict(dim=512), dict(page=20), dict(width=0), dict(stride=3),
                dict(qs=1016), dict(qs=1028), dict(window=-1), dict(first=-1), dict(scale=float("nan")),
                dict(scale=float("inf")), dict(dt=2), dict(fmt=2), dict(batch=2 ** 40), dict(qs=1 << 60),
                dict(width=2 ** 31, stride=2 ** 31), dict(batch=1 << 24), dict(batch=1 << 21, width=1 << 24, stride=1 << 24)):
        assert tree(lib, **bad) == INVALID, bad
    for bad in (dict(q=MIS), dict(out=MIS), dict(kq=MIS), dict(vs=MIS), dict(table=MIS2), dict(context=MIS2),
                dict(sinks=MIS2), dict(mask=MIS4)):
        assert tree(lib, **bad) == MISALIGNED, bad


def test_tree_refuses_an_output_over_q(lib):
    last = 9 * 2 * 2048  # bytes to the last of 10 rows
    for bad in (dict(out=A), dict(q=B, out=ctypes.c_void_p(B.value + last + 2032), qs=2048),
                dict(q=ctypes.c_void_p(B.value + 10 * 8 * 128 * 4 - 16), dt=0), dict(batch=1 << 22, width=1, qh=2, drafts=1)):
        assert tree(lib, **dict(dict(qs=2048, dt=1), **bad)) == INVALID, bad


def tree_workspace(lib, batch, drafts, qh, heads, page, dim, width, window=0, first=0):
    n = ctypes.c_int64(-1)
    code = lib.mxq_tree_attention_workspace(batch, drafts, qh, heads, page, dim, width, window, first, ctypes.byref(n))
    return code, n.value


def test_tree_workspace(lib):
    code, need = tree_workspace(lib, 1, 5, 8, 2, 16, 128, 4096)
    assert code == 0 and need > 0 and need % 4 == 0
    big = dict(batch=1, width=4096, stride=4096, qs=1024)
    assert tree(lib, ws_bytes=need - 1, **big) == INVALID
    assert tree(lib, ws=NULL, ws_bytes=need, **big) == INVALID
    assert tree(lib, ws=MIS, ws_bytes=need, **big) == MISALIGNED
    assert tree_workspace(lib, 1, 5, 8, 2, 16, 128, 1) == (0, 0)  # nothing to split
    assert tree_workspace(lib, 1, 5, 8, 2, 16, 128, 4096, 64)[1] < need  # a window bounds what is split
    assert tree_workspace(lib, 1, 5, 8, 2, 16, 128, 4096, 64, 1 << 40)[1] == need  # first tokens that reach all
    assert tree_workspace(lib, 1, 5, 8, 3, 16, 128, 4096)[0] == INVALID
    assert tree_workspace(lib, 1, 0, 8, 2, 16, 128, 4096)[0] == INVALID
    assert lib.mxq_tree_attention_workspace(1, 5, 8, 2, 16, 128, 4, 0, 0, None) == INVALID


def test_tree_no_device(lib):
    if torch.cuda.device_count() > 0:
        pytest.skip("a GPU is present: this case is only safe without one")
    assert tree(lib) == NOT_SUPPORTED


def test_binding_tree():
    c = mxq.kv_cache(3, 16, 2, 64, device="cpu")
    q, table = torch.zeros(6, 4, 64, dtype=torch.bfloat16), torch.zeros(2, 3, dtype=torch.int32)
    n, m = torch.zeros(2, dtype=torch.int32), torch.zeros(2, 3, 1, dtype=torch.int64)
    for a, t, x, k, kw in ((q[:, :3], table, n, m, {}), (q[:5], table, n, m, {}), (q, table[:1], n, m, {}),
                           (q, table, n[:1], m, {}), (q, table.t().contiguous().t(), n, m, {}),
                           (q[..., :32], table, n, m, {}), (q, table, n, m[..., 0], {}),
                           (q, table, n, torch.zeros(2, 3, 2, dtype=torch.int64), {}),
                           (q, table, n, m, dict(sinks=torch.zeros(3))), (q, table, n, m, {}),
                           (q, table, n, m, dict(out=torch.zeros(6, 4, 32, dtype=torch.bfloat16)))):
        with pytest.raises(ValueError):
            mxq.tree_attention(a, c, t, x, k, **kw)
    for a, t, x, k, kw in ((q.float(), table, n, m, {}), (q, table.long(), n, m, {}), (q, table, n.long(), m, {}),
                           (q, table, n, m.int(), {}), (q, table, n, m, dict(out_dtype=torch.float16)),
                           (q, table, n, m, dict(sinks=torch.zeros(4, dtype=torch.bfloat16)))):
        with pytest.raises(TypeError):
            mxq.tree_attention(a, c, t, x, k, **kw)
    for kw in (dict(window=-1), dict(first=-1)):
        with pytest.raises(mxq.MXQError):
            mxq.tree_attention(q, c, table, n, m, **kw)


def test_tree_mask():
    assert mxq.tree_mask([-1, 0, 0, 1], device="cpu").tolist() == [[[1], [3], [5], [11]]]
    assert mxq.tree_mask(torch.tensor([[-1, 0], [-1, -1]]), device="cpu").tolist() == [[[1], [3]], [[1], [2]]]
    wide = mxq.tree_mask(list(range(-1, 65)), device="cpu")
    assert wide.shape == (1, 66, 2) and wide[0, 63].tolist() == [-1, 0] and wide[0, 65].tolist() == [-1, 3]
    assert mxq.tree_mask([[-1], []], device="cpu").tolist() == [[[1]], [[0]]]
    for bad in ([0], [-1, 1], [-2], [[-1, 0, 5]], []):
        with pytest.raises(ValueError):
            mxq.tree_mask(bad, device="cpu")


# ------------------------------------------------------------------ the draw of a token

def draw(lib, x=A, dt=1, stride=100, rows=3, vocab=100, u=B, t_of=NULL, t=1.0, k_of=NULL, k=0, p_of=NULL, p=1.0, m_of=NULL,
         m=0.0, ws=A, ws_bytes=1 << 40, tokens=C, shares=D):
    return lib.mxq_sample(x, dt, stride, rows, vocab, u, t_of, t, k_of, k, p_of, p, m_of, m, ws, ws_bytes, tokens, shares,
                          NULL)


def test_sample_refusals(lib):
    nan = float("nan")
    for bad in (dict(x=NULL), dict(u=NULL), dict(tokens=NULL), dict(shares=NULL), dict(dt=2), dict(rows=0), dict(rows=-1),
                dict(rows=(1 << 20) + 1), dict(vocab=0), dict(vocab=101), dict(vocab=(1 << 20) + 1, stride=1 << 21),
                dict(stride=1 << 60), dict(t=nan), dict(p=nan), dict(m=nan)):
        assert draw(lib, **bad) == INVALID, bad
    for bad in (dict(x=MIS2, dt=0), dict(x=ctypes.c_void_p(0x1000001)), dict(u=MIS2), dict(t_of=MIS2), dict(k_of=MIS2),
                dict(p_of=MIS2), dict(m_of=MIS2), dict(tokens=MIS2), dict(shares=MIS2)):
        assert draw(lib, **bad) == MISALIGNED, bad
    for bad in (dict(tokens=A), dict(shares=A), dict(tokens=B), dict(shares=B), dict(shares=C), dict(t_of=C), dict(k_of=D),
                dict(p_of=D), dict(m_of=C), dict(tokens=ctypes.c_void_p(A.value + 4 * 296)),
                dict(shares=ctypes.c_void_p(C.value + 8))):
        assert draw(lib, **dict(dict(dt=0), **bad)) == INVALID, bad
    n = ctypes.c_int64(-1)
    assert lib.mxq_sample_workspace(3, 100, ctypes.byref(n)) == 0 and n.value >= 0
    assert lib.mxq_sample_workspace(0, 100, ctypes.byref(n)) == INVALID
    assert lib.mxq_sample_workspace(3, 0, ctypes.byref(n)) == INVALID
    assert lib.mxq_sample_workspace(3, 100, None) == INVALID
    if torch.cuda.device_count() == 0:
        assert draw(lib) == NOT_SUPPORTED
        assert draw(lib, x=MIS2, dt=1, t_of=A, t=nan) == NOT_SUPPORTED


def test_binding_sample():
    x, u = torch.zeros(3, 50), torch.zeros(3)
    for args, kw in (((x[0], u), {}), ((x.t(), u), {}), ((x, u[:2]), {}), ((x, u), dict(temperature=torch.ones(2))),
                     ((x, u), dict(top_k=torch.ones(3, 1, dtype=torch.int32))), ((x, u), dict(tokens=torch.zeros(2, dtype=torch.int32))),
                     ((x, u), {})):  # the last: host tensors
        with pytest.raises(ValueError):
            mxq.sample(*args, **kw)
    for args, kw in (((x.half(), u), {}), ((x.double(), u), {}), ((x, u.double()), {}), ((x, u), dict(top_k=torch.ones(3))),
                     ((x, u), dict(top_p=torch.ones(3, dtype=torch.float64))), ((x, u), dict(tokens=torch.zeros(3))),
                     ((x, u), dict(shares=torch.zeros(3, dtype=torch.bfloat16))), (([1.0], u), {})):
        with pytest.raises(TypeError):
            mxq.sample(*args, **kw)
