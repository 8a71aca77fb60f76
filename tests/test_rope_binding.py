"""What the rotary binding hands to the C calls, without a GPU: the tables of copied and changed
descriptors, and calls that are refused before they reach the library."""
import copy
import ctypes
import gc
import pickle

import numpy as np
import pytest

import context_attention_metadata_gb300 as M


class _Pos:
    """Stands in for the device tensor of positions: the descriptor needs its shape and address."""
    shape = (2, 5)

    @staticmethod
    def data_ptr():
        return 0


def _tables(rope):
    """The frequencies and axes that the C call would read."""
    c = rope._c(_Pos, None, None, 1e-6)
    pairs = c.rot_dim // 2
    return (np.ctypeslib.as_array((ctypes.c_double * pairs).from_address(c.inv_freq)).copy(),
            np.ctypeslib.as_array((ctypes.c_int32 * pairs).from_address(c.axis)).copy())


COPIES = {"deepcopy": copy.deepcopy, "copy": copy.copy,
          "pickle": lambda r: pickle.loads(pickle.dumps(r))}


@pytest.mark.parametrize("how", sorted(COPIES))
def test_a_copy_reads_its_own_tables(how):
    freq, axis = M.rope_frequencies((24, 8), 100.0)
    rope = M.Rope(freq, axis, "adjacent")
    first = rope._c(_Pos, None, None, 1e-6)
    other = COPIES[how](rope)
    c = other._c(_Pos, None, None, 1e-6)
    # arrays of its own: the original's may go at any time
    assert c.inv_freq != first.inv_freq and c.axis != first.axis
    del rope
    gc.collect()
    junk = [np.full(freq.shape, 7.0) for _ in range(64)]  # takes the original's place, if it can
    f, a = _tables(other)
    np.testing.assert_array_equal(f, freq)
    np.testing.assert_array_equal(a, axis)
    assert c.pairing == M.PAIRINGS["adjacent"] and other.rot_dim == 64 and len(junk) == 64


def test_a_changed_descriptor_is_what_the_call_reads():
    rope = M.Rope([1.0, 0.5])
    rope.inv_freq = [3.0, 4.0]
    np.testing.assert_array_equal(_tables(rope)[0], [3.0, 4.0])
    rope.inv_freq[1] = 5.0
    np.testing.assert_array_equal(_tables(rope)[0], [3.0, 5.0])
    rope.axis = [1, 0]
    np.testing.assert_array_equal(_tables(rope)[1], [1, 0])
    for bad in ([1.0], [[1.0, 2.0]]):
        with pytest.raises(ValueError):
            rope.inv_freq = bad
    np.testing.assert_array_equal(_tables(rope)[0], [3.0, 5.0])


class _Tensor:
    """A tensor on the GPU, as far as the binding looks before it makes the call."""
    is_cuda = True

    def __init__(self, torch, shape, dtype):
        self.shape, self.dtype = shape, dtype
        self.base = torch.empty(shape, device="meta")

    def dim(self):
        return len(self.shape)

    def stride(self):
        return self.base.stride()

    def is_contiguous(self):
        return True

    def get_device(self):
        return 0

    def data_ptr(self):
        return 4096


def test_a_closed_plan_is_refused(monkeypatch):
    """A closed plan has no handle, which the C calls take for "no plan": the tokens' order would
    silently stay."""
    import torch
    called = []
    monkeypatch.setattr(M, "_call", lambda name, *args: called.append(name))
    plan = object.__new__(M.Plan)
    plan._h, plan.n = None, 128
    rope = M.Rope([1.0] * 8)
    pos = _Tensor(torch, (1, 128), torch.int32)
    q, dq = (_Tensor(torch, (128, 2, 64), t) for t in (torch.bfloat16, torch.float32))
    out = (_Tensor(torch, (128, 2, 64), torch.bfloat16), None, None)
    stream = type("S", (), {"cuda_stream": 0})()
    with pytest.raises(ValueError, match="closed"):
        M.rope(rope, pos, q, plan=plan, out=out, stream=stream)
    with pytest.raises(ValueError, match="closed"):
        M.rope_bwd(rope, pos, dq, plan=plan, out=out, stream=stream)
    assert called == []
    plan._h = ctypes.c_void_p(1)  # an open one goes through (closing it would free it)
    M.rope(rope, pos, q, plan=plan, out=out, stream=stream)
    M.rope_bwd(rope, pos, dq, plan=plan, out=out, stream=stream)
    assert called == ["marble_rope", "marble_rope_bwd"]
    plan._h = None
