"""Linear attention and page pool entry points: refusals on the host, before any CUDA work
(no GPU needed)."""
import ctypes

import pytest

P = 1 << 20                        # a pointer that is never followed: validation stops first


def _dims(ssd, **kw):
    a = dict(lead=(1, 256), H=8, Hk=2, K=64, V=64, dtype_code=ssd.SSD_DTYPE_BF16)
    later = {k: kw.pop(k) for k in list(kw) if k not in ("lead", "H", "Hk", "K", "V", "dtype_code", "nseq", "strides", "n_pages")}
    a.update(kw)
    d = ssd.linear_attn_dims(**a)
    for k, v in later.items():
        setattr(d, k, v)
    return d


def _fwd(ssd, d, q=P, k=P, v=P, ld=P, init=None, ip=None, cu=None, o=P, fin=None, fp=None):
    return ssd._lib.ssd_linear_attn_fwd(q, k, v, ld, 1.0, init, ip, cu, o, fin, fp, ctypes.byref(d) if d else None, None)


def _update(ssd, d, state=P, q=P, k=P, v=P, ld=P, pages=None, o=P):
    return ssd._lib.ssd_linear_attn_update(state, q, k, v, ld, 1.0, pages, o, ctypes.byref(d) if d else None, None)


@pytest.mark.parametrize("kw,status", [
    (dict(H=6, Hk=4), "UNSUPPORTED"), (dict(K=136), "UNSUPPORTED"), (dict(V=256), "UNSUPPORTED"), (dict(K=12), "UNSUPPORTED"),
    (dict(V=4), "UNSUPPORTED"), (dict(H=0), "INVALID_ARG"), (dict(Hk=0), "INVALID_ARG"), (dict(K=-8), "INVALID_ARG"),
    (dict(dtype_code=7), "INVALID_ARG"), (dict(strides=(8 * 64 - 8, 0, 0)), "INVALID_ARG"),
    (dict(strides=(0, 2 * 64 + 4, 0)), "UNSUPPORTED"), (dict(strides=(0, 0, 1 << 31)), "UNSUPPORTED"),
    (dict(H=65536, Hk=1), "UNSUPPORTED"),
])
def test_bad_geometry(ssd, kw, status):
    d = _dims(ssd, **kw)
    want = getattr(ssd, "SSD_ERR_" + status)
    assert _fwd(ssd, d) == want and ssd._lib.ssd_last_error().decode()
    with pytest.raises(ssd.SSDError, match=status):
        ssd.linear_attn_workspace_size(d)
    d.seqlen = 1
    assert _update(ssd, d) == want


@pytest.mark.parametrize("kw", [dict(batch=-1), dict(seqlen=-1), dict(batch=1 << 40, seqlen=1 << 40)])
def test_bad_dense_sizes(ssd, kw):
    assert _fwd(ssd, _dims(ssd, **kw)) in (ssd.SSD_ERR_INVALID_ARG, ssd.SSD_ERR_UNSUPPORTED)


def test_too_many_tokens(ssd):
    assert _fwd(ssd, _dims(ssd, lead=(1, 1 << 31))) == ssd.SSD_ERR_UNSUPPORTED
    assert _fwd(ssd, _dims(ssd, lead=(1 << 31,), nseq=1), cu=P) == ssd.SSD_ERR_UNSUPPORTED


@pytest.mark.parametrize("kw", [dict(q=None), dict(k=None), dict(v=None), dict(o=None), dict(ld=None), dict(q=P + 2), dict(v=P + 8),
                                dict(o=P + 8), dict(init=P + 4), dict(fin=P + 8), dict(ld=P + 1), dict(ip=P), dict(fp=P),
                                dict(init=P, ip=P), dict(fin=P, fp=P), dict(init=P, ip=P + 2), dict(cu=P + 1)])
def test_bad_pointers(ssd, kw):
    assert _fwd(ssd, _dims(ssd), **kw) == ssd.SSD_ERR_INVALID_ARG        # page lists: n_pages is 0


@pytest.mark.parametrize("kw", [dict(state=None), dict(q=None), dict(k=None), dict(v=None), dict(o=None), dict(ld=None),
                                dict(state=P + 8), dict(k=P + 4), dict(pages=P), dict(pages=P + 2)])
def test_bad_update_pointers(ssd, kw):
    assert _update(ssd, _dims(ssd, lead=(4, 1)), **kw) == ssd.SSD_ERR_INVALID_ARG


def test_null_dims_and_update_of_more_than_one_token(ssd):
    assert _fwd(ssd, None) == ssd.SSD_ERR_INVALID_ARG and _update(ssd, None) == ssd.SSD_ERR_INVALID_ARG
    assert _update(ssd, _dims(ssd, lead=(4, 2))) == ssd.SSD_ERR_INVALID_ARG
    assert ssd._lib.ssd_linear_attn_fwd_workspace_size(ctypes.byref(_dims(ssd)), None) == ssd.SSD_ERR_INVALID_ARG


def test_small_or_misaligned_workspace(ssd):
    d = _dims(ssd, lead=(300,), nseq=3)
    need = ssd.linear_attn_workspace_size(d)
    assert need >= 256
    d.workspace, d.workspace_bytes = P, need - 1
    assert _fwd(ssd, d, cu=P) == ssd.SSD_ERR_INVALID_ARG
    d.workspace, d.workspace_bytes = P + 16, need
    assert _fwd(ssd, d, cu=P) == ssd.SSD_ERR_INVALID_ARG


def test_workspace_holds_the_states_of_the_segments(ssd):
    state = 64 * 64 * 64 * 4                            # 64 heads of [64][64] floats
    f32 = dict(H=64, Hk=64, dtype_code=ssd.SSD_DTYPE_F32)
    # fp32, 64 sequences: CTAs for every SM without cutting a sequence, so nothing but the four
    # 256-byte pieces of a packed call without sequences
    assert ssd.linear_attn_workspace_size(_dims(ssd, lead=(64, 512), **f32)) == 4 * 256
    # bf16: a state per segment and one per sequence
    assert ssd.linear_attn_workspace_size(_dims(ssd, lead=(64, 512), H=64, Hk=64)) == 64 * 2 * state
    ssd.set_segment_tokens(128)
    try:
        for kw in (f32, dict(H=64, Hk=64)):
            assert ssd.linear_attn_workspace_size(_dims(ssd, lead=(64, 512), **kw)) == 64 * 5 * state
    finally:
        ssd.set_segment_tokens(0)


def _pool(ssd, **kw):
    arrays, sizes = (ctypes.c_void_p * 2)(P, P), (ctypes.c_int64 * 2)(64, 7)
    a = dict(n_pages=8, n_rows=4, max_pages=2, n_arrays=2, arrays=arrays, page_bytes=sizes, refcount=P, table=P, length=P, live=P)
    a.update(kw)
    c = ssd.SSDPagePool(**a)
    c._keep = (arrays, sizes)
    return c


@pytest.mark.parametrize("kw,status", [
    (dict(n_pages=0), "INVALID_ARG"), (dict(n_rows=0), "INVALID_ARG"), (dict(max_pages=0), "INVALID_ARG"),
    (dict(n_pages=(1 << 20) + 1), "UNSUPPORTED"), (dict(n_rows=(1 << 20) + 1), "UNSUPPORTED"),
    (dict(n_arrays=-1), "INVALID_ARG"), (dict(n_arrays=129), "UNSUPPORTED"), (dict(arrays=None), "INVALID_ARG"),
    (dict(page_bytes=None), "INVALID_ARG"), (dict(refcount=None), "INVALID_ARG"), (dict(table=None), "INVALID_ARG"),
    (dict(length=None), "INVALID_ARG"), (dict(live=None), "INVALID_ARG"), (dict(refcount=P + 2), "INVALID_ARG"),
    (dict(arrays=(ctypes.c_void_p * 2)(P, None)), "INVALID_ARG"), (dict(page_bytes=(ctypes.c_int64 * 2)(64, 0)), "INVALID_ARG"),
    (dict(page_bytes=(ctypes.c_int64 * 2)(64, 1 << 50)), "UNSUPPORTED"),
    (dict(workspace=P, workspace_bytes=8), "INVALID_ARG"), (dict(workspace=P + 4, workspace_bytes=1 << 20), "INVALID_ARG"),
])
def test_bad_pools(ssd, kw, status):
    c = _pool(ssd, **kw)
    r, want = ctypes.byref(c), getattr(ssd, "SSD_ERR_" + status)
    lib = ssd._lib
    calls = [lib.ssd_pages_append(r, P, 1, 0, None), lib.ssd_pages_fork(r, P, P, 1, None), lib.ssd_pages_free(r, P, 1, None),
             lib.ssd_pages_copy(r, P, P, 1, None), lib.ssd_pages_compact(r, P, P, None)]
    assert calls == [want] * 5
    assert lib.ssd_last_error().decode()


def test_bad_page_lists(ssd):
    r, lib, bad = ctypes.byref(_pool(ssd)), ssd._lib, ssd.SSD_ERR_INVALID_ARG
    assert lib.ssd_pages_append(r, None, 1, 0, None) == bad
    assert lib.ssd_pages_append(r, P, -1, 0, None) == bad
    assert lib.ssd_pages_append(r, P + 2, 1, 0, None) == bad
    assert lib.ssd_pages_fork(r, P, None, 1, None) == bad
    assert lib.ssd_pages_copy(r, None, P, 1, None) == bad
    assert lib.ssd_pages_compact(r, None, P, None) == bad
    assert lib.ssd_pages_compact(r, P, P + 1, None) == bad
    assert lib.ssd_pages_append(None, P, 1, 0, None) == bad
    for n in (0,):                                      # nothing asked for: nothing launched
        assert lib.ssd_pages_append(r, None, n, 0, None) == ssd.SSD_OK and lib.ssd_last_launch_count() == 0
    size = ctypes.c_size_t(0)
    assert lib.ssd_pages_workspace_size(r, 5, None) == bad
    assert lib.ssd_pages_workspace_size(r, 100, ctypes.byref(size)) == ssd.SSD_OK and size.value >= 3 * 4 * 100


def test_binding_checks_before_the_library(ssd):
    import torch
    z = torch.zeros(2, 4, 16)
    with pytest.raises(ValueError, match="must be on"):
        ssd.linear_attn_update(torch.zeros(2, 4, 16, 16), z, z, z, torch.zeros(4))
    with pytest.raises(ValueError, match="array 0"):
        ssd.PagePool([z], 2, 2)


class _OnDevice:
    """The layout of a CPU tensor, as the binding's checks would see it on a device."""
    is_cuda = True

    def __init__(self, t):
        self.t, self.shape, self.dtype, self.device = t, t.shape, t.dtype, t.device

    def stride(self):
        return self.t.stride()

    def is_contiguous(self):
        return self.t.is_contiguous()


def test_token_strides(ssd):
    """Expanded (stride 0) and overlapping tokens are refused: the library reads a stride of 0
    as "contiguous"."""
    import torch
    H, K = 4, 16
    step = lambda t: ssd._token_stride(_OnDevice(t), "q", t.shape[:-2], H, K, t.dtype, t.device)  # noqa: E731
    one = torch.zeros(1, H, K)
    for t in (one.expand(7, H, K), one.expand(2, 7, H, K), one.expand(1, 7, H, K), one[None].expand(5, 1, H, K),
              torch.zeros(7 * H * K).as_strided((3, H, K), (H * K - 8, K, 1)),
              torch.zeros(7 * H * K).as_strided((2, 3, H, K), (3 * K, K, K, 1))):
        with pytest.raises(ValueError, match="share memory"):
            step(t)
    with pytest.raises(ValueError, match="without a gap"):
        step(torch.zeros(1, 7, H, K).expand(2, 7, H, K))
    row = torch.zeros(14, H * K + 8)[:, :H * K].unflatten(1, (H, K))
    assert step(row) == H * K + 8 and step(row.unflatten(0, (2, 7))) == H * K + 8
    assert step(row.unflatten(0, (14, 1))) == H * K + 8
    for t in (one.expand(1, 1, H, K), one, torch.zeros(0, H, K), torch.zeros(2, 0, H, K), torch.zeros(3, 7, H, K)):
        assert step(t) == H * K


def test_one_array_with_one_page_list_holds_every_sequence(ssd):
    """The side without a list names states 0 .. nseq-1 of an array of n_pages."""
    for kw in (dict(ip=P), dict(fp=P)):
        d = _dims(ssd, lead=(4, 256), n_pages=3)
        assert _fwd(ssd, d, init=P, fin=P, **kw) == ssd.SSD_ERR_INVALID_ARG
        assert b"more sequences" in ssd._lib.ssd_last_error()
