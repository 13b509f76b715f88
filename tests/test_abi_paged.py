"""The entry points of rotary positions and the paged cache on the CPU: what
they refuse before anything touches a device, in the library and in the
binding."""
import ctypes as C
import os

import pytest


@pytest.fixture(scope="module")
def dq():
    import dynamic_quantized_gemm_amd as dq
    from dynamic_quantized_gemm_amd import build

    if not os.path.exists(dq.LIB_PATH):
        build.build()
    dq.load()
    return dq


def test_rope_init_refuses(dq):
    lib = dq.load()

    def init(dim=8, rot=8, axis=(0, 0, 0, 0), freq=(1.0, 0.1, 0.01, 0.001)):
        h = C.c_void_p()
        a = None if axis is None else C.cast((C.c_int32 * len(axis))(*axis), C.c_void_p)
        f = None if freq is None else C.cast((C.c_double * len(freq))(*freq), C.c_void_p)
        rc = lib.dq_rope_init(C.byref(h), dim, rot, a, f, 0)
        assert h.value is None and dq.dqip_last_error()
        return rc

    assert init(dim=7) == dq.DQ_ERR_ARG
    assert init(rot=0) == dq.DQ_ERR_ARG
    assert init(rot=10) == dq.DQ_ERR_ARG
    assert init(rot=7) == dq.DQ_ERR_ARG
    assert init(dim=dq.DQ_ROPE_DIM_MAX + 2) == dq.DQ_ERR_RANGE
    assert init(axis=None) == dq.DQ_ERR_ARG
    assert init(freq=None) == dq.DQ_ERR_ARG
    assert init(axis=(0, 1, -1, 0)) == dq.DQ_ERR_RANGE
    assert init(axis=(0, 1, dq.DQ_ROPE_AXES_MAX, 0)) == dq.DQ_ERR_RANGE
    assert init(freq=(1.0, float("nan"), 1.0, 1.0)) == dq.DQ_ERR_ARG
    assert init(freq=(1.0, 1e10, 1.0, 1.0)) == dq.DQ_ERR_ARG
    assert lib.dq_rope_init(None, 8, 8, None, None, 0) == dq.DQ_ERR_ARG
    with pytest.raises(dq.DQError):
        dq.dq_rope_init(8, 8, [0, 0, 0], [1.0] * 4)


def test_kv_init_refuses(dq):
    lib = dq.load()

    def init(batch=2, hq=8, hk=2, dim=64, pages=16, size=16, per=8, qt=dq.DQ_BF16, ct=dq.DQ_I8):
        h = C.c_void_p()
        rc = lib.dq_kv_init(C.byref(h), batch, hq, hk, dim, pages, size, per, qt, ct, 0)
        assert h.value is None and dq.dqip_last_error()
        return rc

    for name in ("batch", "hq", "hk", "pages", "size", "per"):
        assert init(**{name: 0}) == dq.DQ_ERR_ARG
        assert init(**{name: -5}) == dq.DQ_ERR_ARG
    assert init(hq=9) == dq.DQ_ERR_ARG
    assert init(dim=0) == dq.DQ_ERR_ARG
    assert init(dim=72) == dq.DQ_ERR_ARG
    assert init(dim=dq.DQ_KV_DIM_MAX + 16) == dq.DQ_ERR_RANGE
    assert init(qt=dq.DQ_I8) == dq.DQ_ERR_TYPE
    assert init(ct=dq.DQ_F32) == dq.DQ_ERR_TYPE
    assert init(ct=dq.DQ_U8) == dq.DQ_ERR_TYPE
    assert init(batch=65536, hk=1) == dq.DQ_ERR_RANGE
    assert init(batch=40000) == dq.DQ_ERR_RANGE                 # 80000 heads
    assert init(size=1 << 20, per=1 << 11) == dq.DQ_ERR_RANGE   # 2^31 slots of a sequence
    assert init(pages=1 << 26) == dq.DQ_ERR_RANGE               # 2^31 rows
    assert init(pages=2 ** 31 - 1, size=2 ** 31 - 1, per=1, hq=2 ** 31 - 1, hk=2 ** 31 - 1) == dq.DQ_ERR_RANGE
    assert lib.dq_kv_init(None, 2, 8, 2, 64, 16, 16, 8, 1, 2, 0) == dq.DQ_ERR_ARG


def test_null_contexts(dq):
    lib = dq.load()
    assert lib.dq_rope_forward(None, 1, 0, 1, 1, 8, 8, 1, 1, 8, 8, 0, None) == dq.DQ_ERR_STATE
    assert lib.dq_kv_append(None, 1, 1, 8, 8, 1, 8, 8, 1, None, 1, 1, 1, None, None, None, 0, 0, None, None, None,
                            None) == dq.DQ_ERR_STATE
    assert lib.dq_kv_read(None, 1, 1, None, 1, 1, 1, None, None, 1, 1, None) == dq.DQ_ERR_STATE
    assert lib.dq_kv_attend(None, 1, 1, 8, 8, 1, 1, 1, 1, None, None, 1, 1.0, None, 0, None, None, 1.0,
                            None) == dq.DQ_ERR_STATE
    assert lib.dq_kv_evict(None, 1, 1, 0, 0, 1, 1, 1, 1, 1, 1, 1, None, None, 1, 1, 1, None) == dq.DQ_ERR_STATE
    n = C.c_int()
    assert lib.dq_kv_take_errors(None, C.byref(n), None) == dq.DQ_ERR_STATE
    assert lib.dq_rope_info(None) is None and lib.dq_kv_info(None) is None
    lib.dq_rope_release(None)
    lib.dq_kv_release(None)


class _Fake:
    """A device tensor as the binding's checks see it; its memory is never
    asked for unless every check has passed."""

    def __init__(self, shape, elem=2, stride=None, device="cuda"):
        self.shape, self._e = tuple(shape), elem
        dense = []
        for i in range(len(shape)):
            n = 1
            for d in shape[i + 1:]:
                n *= d
            dense.append(n)
        self._s, self._dense = tuple(stride or dense), tuple(dense)
        self.device = type("D", (), {"type": device})()
        self.is_cuda = device == "cuda"
        self.dtype = "torch.bfloat16"

    def stride(self):
        return self._s

    def numel(self):
        n = 1
        for d in self.shape:
            n *= d
        return n

    def element_size(self):
        return self._e

    @property
    def nbytes(self):
        return self.numel() * self._e

    def is_contiguous(self):
        return self._s == self._dense

    def data_ptr(self):
        return 1 << 20


class _Reached(Exception):
    pass


@pytest.fixture
def bound(dq, monkeypatch):
    """Contexts as the binding records them, and a library that only says that
    a call has passed the checks."""
    b = dq._binding
    rope, kv = 0xdead1000, 0xdead2000
    monkeypatch.setitem(b._ROPE_DIMS, rope, (64, 3))
    rows = 16 * 2 * 8
    monkeypatch.setitem(b._KV_DIMS, kv, (4, 6, 2, 64, 5, 40, 2, rows * 64, 4 * rows))

    class Lib:
        def __getattr__(self, name):
            def call(*a):
                raise _Reached(name)
            return call

    monkeypatch.setattr(b, "load", lambda: Lib())
    return rope, kv


def _refused(dq, call, **change):
    with pytest.raises(dq.DQError) as e:
        call(**change)
    assert e.value.status in (dq.DQ_ERR_ARG, dq.DQ_ERR_STATE, dq.DQ_ERR_TYPE)


def test_binding_refuses_rope_tensors(dq, bound):
    rope, _ = bound

    def call(ctx=rope, x=_Fake((7, 3, 64), stride=(1000, 64, 1)), pos=_Fake((3, 7), 4), y=_Fake((7, 3, 64)), **k):
        dq.dq_rope_forward(ctx, x, pos, y, stream=0, **k)

    with pytest.raises(_Reached):
        call()
    _refused(dq, call, ctx=5)
    for bad in (_Fake((7, 3, 32)), _Fake((7, 192)), _Fake((7, 3, 64), stride=(192, 64, 2)), _Fake((7, 3, 64), 4),
                _Fake((7, 3, 64), device="cpu")):
        _refused(dq, call, x=bad)
        _refused(dq, call, y=bad)
    _refused(dq, call, y=_Fake((6, 3, 64)))
    _refused(dq, call, y=_Fake((7, 4, 64)))
    _refused(dq, call, pos=_Fake((2, 7), 4))
    _refused(dq, call, pos=_Fake((3, 7), 4, stride=(8, 1)))


def test_binding_refuses_cache_tensors(dq, bound):
    rope, kv = bound
    cache = dict(block_table=_Fake((4, 5), 4), k_cache=_Fake((16, 2, 8, 64), 1), v_cache=_Fake((16, 2, 8, 64), 1),
                 k_scale=_Fake((16, 2, 8), 4), v_scale=_Fake((16, 2, 8), 4))
    short = dict(block_table=_Fake((3, 5), 4), k_cache=_Fake((15, 2, 8, 64), 1), v_cache=_Fake((16, 2, 7, 64), 1),
                 k_scale=_Fake((16, 2, 7), 4), v_scale=_Fake((16, 8, 2), 2))
    n = 9

    def append(**k):
        a = dict(k=_Fake((n, 2, 64), stride=(640, 64, 1)), v=_Fake((n, 2, 64)), index=_Fake((n,), 4), **cache)
        a.update(seq_ids=_Fake((n,), 4), q=_Fake((n, 6, 64)), q_out=_Fake((n, 6, 64)), rope=rope,
                 positions=_Fake((3, n), 4))
        a.update(k)
        dq.dq_kv_append(a.pop("ctx", kv), stream=0, **a)

    def read(**k):
        a = dict(index=_Fake((n,), 4), seq_ids=_Fake((n,), 4), k_out=_Fake((n, 2, 64)), v_out=_Fake((n, 2, 64)),
                 **cache)
        a.update(k)
        dq.dq_kv_read(a.pop("ctx", kv), stream=0, **a)

    def attend(**k):
        a = dict(q=_Fake((4, 6, 64)), lens=_Fake((4,), 4), out=_Fake((4, 6, 64)), sm_scale=0.1, lse=_Fake((4, 6), 4),
                 scores=_Fake((4, 2, 40), 4), scores_out=_Fake((4, 2, 40), 4), **cache)
        a.update(k)
        dq.dq_kv_attend(a.pop("ctx", kv), stream=0, **a)

    def evict(**k):
        a = dict(budget=8, lens=_Fake((4,), 4), newest=_Fake((4,), 4), lens_out=_Fake((4,), 4), **cache)
        for name in ("scores", "order", "scores_out", "order_out"):
            a[name] = _Fake((4, 2, 40), 4)
        a.update(k)
        dq.dq_kv_evict(a.pop("ctx", kv), stream=0, **a)

    for call in (append, read, attend, evict):
        with pytest.raises(_Reached):
            call()
        _refused(dq, call, ctx=6)
        for name in cache:
            _refused(dq, call, **{name: short[name]})
            _refused(dq, call, **{name: _Fake(cache[name].shape, cache[name].element_size(), device="cpu")})
    for name in ("k", "v"):
        for bad in (_Fake((n, 2, 32)), _Fake((n, 3, 64)), _Fake((n, 2, 64), 4), _Fake((n, 2, 64), stride=(128, 1, 2))):
            _refused(dq, append, **{name: bad})
    _refused(dq, append, v=_Fake((n - 1, 2, 64)))
    _refused(dq, append, index=_Fake((n - 1,), 4))
    _refused(dq, append, seq_ids=_Fake((n - 1,), 4))
    _refused(dq, append, q=_Fake((n, 5, 64)))
    _refused(dq, append, q_out=_Fake((n, 5, 64)))
    _refused(dq, append, positions=_Fake((2, n), 4))
    _refused(dq, append, rope=None)
    _refused(dq, append, rope=7)
    _refused(dq, read, k_out=_Fake((n, 2, 63)))
    _refused(dq, read, v_out=_Fake((n, 2, 63)))
    _refused(dq, read, seq_ids=_Fake((n - 1,), 4))
    _refused(dq, attend, q=_Fake((4, 5, 64)))
    _refused(dq, attend, lens=_Fake((3,), 4))
    _refused(dq, attend, out=_Fake((3, 6, 64)))
    _refused(dq, attend, lse=_Fake((4, 5), 4))
    _refused(dq, attend, scores=_Fake((4, 2, 39), 4))
    _refused(dq, attend, scores_out=_Fake((4, 2, 39), 4))
    for name in ("scores", "order", "scores_out", "order_out"):
        _refused(dq, evict, **{name: _Fake((4, 2, 39), 4)})
    _refused(dq, evict, newest=_Fake((3,), 4))
    _refused(dq, evict, lens_out=_Fake((3,), 4))
