"""The binding of rotary positions and the paged cache refuses tensors of
another type than the kernels would read, before anything touches a device:
64-bit integers where 32 bits are read, and the floating point types for one
another."""
import pytest
import torch

from test_abi_paged import _Fake, _Reached, dq  # noqa: F401

F32, BF16, F16, I8 = torch.float32, torch.bfloat16, torch.float16, torch.int8
I32, I64 = torch.int32, torch.int64
N = 9


def _tensor(dtype, *shape):
    t = _Fake(shape, dtype.itemsize)
    t.dtype = dtype
    return t


@pytest.fixture
def bound(dq, monkeypatch):  # noqa: F811
    """Contexts as the binding records them for bf16 queries on an int8 cache,
    and a library that only says that a call has passed the checks."""
    b = dq._binding
    rope, kv = 0xdead3000, 0xdead4000
    rows = 16 * 2 * 8
    monkeypatch.setitem(b._ROPE_DIMS, rope, (64, 3))
    monkeypatch.setitem(b._KV_DIMS, kv, (4, 6, 2, 64, 5, 40, 2, rows * 64, 4 * rows))
    monkeypatch.setitem(b._KV_TYPES, kv, (dq.DQ_BF16, dq.DQ_I8))

    class Lib:
        def __getattr__(self, name):
            def call(*a):
                raise _Reached(name)
            return call

    monkeypatch.setattr(b, "load", lambda: Lib())
    return rope, kv


def _calls(dq, bound):  # noqa: F811
    """name -> (call, its tensors)."""
    rope, kv = bound
    cache = dict(block_table=_tensor(I32, 4, 5), k_cache=_tensor(I8, 16, 2, 8, 64), v_cache=_tensor(I8, 16, 2, 8, 64),
                 k_scale=_tensor(F32, 16, 2, 8), v_scale=_tensor(F32, 16, 2, 8))
    state = dict(scores=_tensor(F32, 4, 2, 40), scores_out=_tensor(F32, 4, 2, 40))
    rows, heads = _tensor(BF16, N, 2, 64), _tensor(BF16, N, 6, 64)
    q, out = _tensor(BF16, 4, 6, 64), _tensor(BF16, 4, 6, 64)
    return {
        "rope": (lambda **a: dq.dq_rope_forward(rope, a["x"], a["positions"], a["y"], stream=0),
                 dict(x=_tensor(BF16, N, 3, 64), positions=_tensor(I32, 3, N), y=_tensor(BF16, N, 3, 64))),
        "append": (lambda **a: dq.dq_kv_append(kv, rope=rope, stream=0, **a),
                   dict(k=rows, v=rows, index=_tensor(I32, N), seq_ids=_tensor(I32, N), q=heads, q_out=heads,
                        positions=_tensor(I32, 3, N), **cache)),
        "read": (lambda **a: dq.dq_kv_read(kv, stream=0, **a),
                 dict(index=_tensor(I32, N), seq_ids=_tensor(I32, N), k_out=rows, v_out=rows, **cache)),
        "attend": (lambda **a: dq.dq_kv_attend(kv, sm_scale=0.1, stream=0, **a),
                   dict(q=q, lens=_tensor(I32, 4), out=out, lse=_tensor(F32, 4, 6), **cache, **state)),
        "evict": (lambda **a: dq.dq_kv_evict(kv, 8, stream=0, **a),
                  dict(lens=_tensor(I32, 4), newest=_tensor(I32, 4), order=_tensor(I32, 4, 2, 40),
                       order_out=_tensor(I32, 4, 2, 40), lens_out=_tensor(I32, 4), **cache, **state)),
    }


@pytest.mark.parametrize("name", ["rope", "append", "read", "attend", "evict"])
def test_refuses_other_types(dq, bound, name):  # noqa: F811
    call, tensors = _calls(dq, bound)[name]
    with pytest.raises(_Reached):
        call(**tensors)
    with pytest.raises(_Reached):  # and once more, by the checks' short way
        call(**tensors)
    for which, t in tensors.items():
        others = {I32: (I64, F32, torch.int16), F32: (torch.float64, I32, BF16), I8: (BF16, I32),
                  BF16: (F16, F32)}[t.dtype]
        if name == "rope" and which == "x":
            others = (I8, I64)  # (x's type is the call's)
        for other in others:
            with pytest.raises(dq.DQError) as e:
                call(**{**tensors, which: _tensor(other, *t.shape)})
            assert e.value.status in (dq.DQ_ERR_TYPE, dq.DQ_ERR_ARG), (which, other)


def test_takes_views_of_the_same_bytes(dq, bound):  # noqa: F811
    """A dtype that the calls do not know is taken by the size of its
    elements, as a view of a cache's or an index's bytes is."""
    for name, which, dtype in (("attend", "k_cache", torch.uint8), ("append", "v_cache", torch.uint8),
                               ("append", "q_out", torch.int16), ("attend", "q", torch.int16)):
        call, tensors = _calls(dq, bound)[name]
        with pytest.raises(_Reached):
            call(**{**tensors, which: _tensor(dtype, *tensors[which].shape)})


def test_rope_output_has_the_inputs_type(dq, bound):  # noqa: F811
    call, tensors = _calls(dq, bound)["rope"]
    for t in (F32, F16):
        x = _tensor(t, *tensors["x"].shape)
        with pytest.raises(dq.DQError):
            call(**{**tensors, "x": x})
        with pytest.raises(_Reached):
            call(**{**tensors, "x": x, "y": _tensor(t, *x.shape)})


def test_rope_refuses_types_that_do_not_exist(dq, bound):  # noqa: F811
    rope, _ = bound
    x, pos = _tensor(BF16, N, 3, 64), _tensor(I32, 3, N)
    for code in (-1, 5, 6, 99):
        with pytest.raises(dq.DQError) as e:
            dq.dq_rope_forward(rope, x, pos, x, type_=code, stream=0)
        assert e.value.status == dq.DQ_ERR_TYPE
