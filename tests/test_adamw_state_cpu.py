"""What an AdamW state takes for its parameters and buffers, on a host without a GPU (nothing is launched).

The checks are the binding's own but for the device: these tensors are on the CPU.
"""

import pytest
import torch

import ragged_grouped_gemm_histogram_amd as moe

BF16, F32 = torch.bfloat16, torch.float32


@pytest.fixture(autouse=True)
def any_device(monkeypatch):
    def want(t, name, dtype, shape, device):
        if not isinstance(t, torch.Tensor) or t.dtype != dtype:
            raise TypeError(f"{name}: type")
        if tuple(t.shape) != tuple(shape) or not t.is_contiguous():
            raise ValueError(f"{name}: shape or strides")
        return t

    monkeypatch.setattr(moe, "_want", want)


def state(*shapes, dtype=F32, **kw):
    return moe.moe_adamw_state([torch.nn.Parameter(torch.zeros(s, dtype=dtype)) for s in shapes], **kw)


def test_a_parameter_that_became_a_transposed_view_is_refused():
    s = state((4, 4), (8, 3))
    s._take_params()
    s.params[0].data = s.params[0].data.t()  # the same address, values and shape
    with pytest.raises(ValueError, match=r"params\[0\]"):
        s._take_params()
    s.params[0].data = s.params[0].data.t()
    s._take_params()
    s.params[1].data = s.params[1].data.t()
    with pytest.raises(ValueError, match=r"params\[1\]"):
        s._take_params()


@pytest.mark.parametrize("old,new", [(F32, BF16), (BF16, F32), (BF16, torch.float16), (F32, torch.int32)])
def test_a_parameter_whose_type_changed_at_its_address_is_refused(old, new):
    memory = torch.zeros(64, dtype=F32)
    s = moe.moe_adamw_state([torch.zeros(8), memory.view(old)[:32]])
    s._take_params()
    s.params[1] = memory.view(new)[:32]
    with pytest.raises(TypeError, match=r"params\[1\]"):
        s._take_params()


def test_parameters_that_are_as_they_were_or_moved_are_taken():
    s = state((4, 4), (0,), (8, 3), dtype=BF16)
    s._take_params()
    s.params[2].data = s.params[2].data.clone()
    s._take_params()
    assert list(s._param_ptrs) == [p.data_ptr() for p in s.params]


@pytest.mark.parametrize("change", [lambda p: p.append(torch.zeros(4)), lambda p: p.pop(), lambda p: p.clear()])
def test_another_number_of_parameters_is_refused(change):
    s = state((4, 4), (8, 3))
    change(s.params)
    with pytest.raises(ValueError, match="2 parameters"):
        s._take_params()


def test_gradients_that_are_no_tensors_are_named():
    s = state((4, 4), (8, 3))
    for bad in (None, [1.0], 3):
        with pytest.raises(TypeError, match=r"grads\[1\]"):
            s._take_grads([torch.zeros(4, 4), bad])


def blocks(memory, at):
    """8-bit moments of 64 values in 66 bytes of `memory`."""
    return moe.Blocks8(memory[at:at + 64], memory[at + 64:at + 66])


def test_buffers_that_share_memory_are_refused():
    p, m = [torch.zeros(64)], torch.zeros(256)
    apart = (m[:64], m[64:128], m[128:192])
    moe.AdamW(p, *apart)
    for args in ((m[:64], m[:64]), (m[:64], m[32:96]), (m[:64], m[64:128], m[64:128]), (m[:64], m[64:128], m[127:191]),
                 (p[0], m[:64]), (m[:64], p[0]), (m[:64], m[64:128], p[0])):
        with pytest.raises(ValueError, match="share memory"):
            moe.AdamW(p, *args)
    b = torch.zeros(192, dtype=torch.uint8)
    moe.AdamW(p, blocks(b, 0), blocks(b, 66))
    for args in ((blocks(b, 0), blocks(b, 0)), (blocks(b, 0), blocks(b, 65)),
                 (moe.Blocks8(b[:64], b[64:66]), moe.Blocks8(b[66:130], b[64:66])),
                 (blocks(b, 0), blocks(b, 66), b.new_zeros(256).view(F32)[:64])):
        if len(args) == 3:  # (apart: taken)
            moe.AdamW(p, *args)
            continue
        with pytest.raises(ValueError, match="share memory"):
            moe.AdamW(p, *args)


def test_buffers_that_come_to_share_memory_are_refused():
    s = state((64,), (8, 3), master=True)
    s._take_params()
    m, master = s.exp_avg, s.master
    s.exp_avg = s.exp_avg_sq
    with pytest.raises(ValueError, match="share memory"):
        s._take_params()
    with pytest.raises(ValueError, match="share memory"):  # and again
        s._take_params()
    s.exp_avg = m
    s._take_params()
    s.params[0].data = master[:64]
    with pytest.raises(ValueError, match="share memory"):
        s._take_params()
    # all at once: what was a moment's memory is a parameter's now
    s.params[0].data, s.exp_avg = s.exp_avg[:64], torch.zeros(96)
    s._take_params()
