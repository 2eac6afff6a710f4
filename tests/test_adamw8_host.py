"""The host side of the step with moments in 8 bits: what the list and the C calls refuse, without a GPU."""
import ctypes

import pytest
import torch

from tensor_grad_clip_gb300 import SomaOpt, TensorList, _abi, build, from_8bit, to_8bit, zeros_8bit

P = 1 << 20
F8 = torch.float8_e4m3fn


@pytest.fixture(scope="module", autouse=True)
def lib():
    build.build()
    return _abi.load()


def entry(**kw):
    e = _abi.soma_tensor_t()
    e.param, e.grad, e.exp_avg, e.exp_avg_sq, e.param_lowp = P, 2 * P, 3 * P, 4 * P, None
    e.numel, e.group, e.grad_dtype, e.trainable, e.owned, e.lowp_dtype = 8, 0, 0, 1, 1, 0
    for k, v in kw.items():
        setattr(e, k, v)
    return e


def step(entries, scales, n=None, call="soma_opt_step8"):
    opt = SomaOpt(0)
    opt.add_group(lr=1e-3)
    arr = (_abi.soma_tensor_t * len(entries))(*entries)
    sc = None if scales is None else (_abi.soma_scales_t * len(scales))(*scales)
    st = getattr(_abi, call)(opt.handle, arr, sc, len(entries) if n is None else n, 1.0, 1.0, None)
    return st, _abi.soma_opt_last_error(opt.handle).decode()


@pytest.mark.parametrize("call", ["soma_opt_step8", "soma_opt_step_graph8"])
def test_refusals(call):
    good = (5 * P, 6 * P)
    for entries, scales, status, word in (
            ([entry()], None, 1, "scales is NULL"),
            ([entry()], [(5 * P, None)], 1, "one of the two"),
            ([entry(), entry()], [good, (None, 6 * P)], 1, "scales[1]"),
            ([entry()], [(5 * P + 2, 6 * P)], _abi.SOMA_ERR_ALIGNMENT, "aligned"),
            ([entry()], [(5 * P, 6 * P + 1)], _abi.SOMA_ERR_ALIGNMENT, "aligned"),
            ([entry(param=P + 2)], [good], _abi.SOMA_ERR_ALIGNMENT, "aligned"),
            ([entry(exp_avg=3 * P + 1)], [(None, None)], _abi.SOMA_ERR_ALIGNMENT, "aligned"),  # fp32 moments
            ([entry(exp_avg=None)], [good], 1, "null buffer"),
            ([entry(group=3)], [good], _abi.SOMA_ERR_BAD_GROUP, "group"),
            ([entry(grad_dtype=7)], [good], _abi.SOMA_ERR_DTYPE, "grad_dtype")):
        st, text = step(entries, scales, call=call)
        assert st == status and word in text, (st, text, word)
    st, text = step([entry()], [good], n=-1, call=call)
    assert st == 1 and "n < 0" in text


def test_dead_handles():
    assert _abi.soma_opt_step8(None, None, None, 0, 1.0, 1.0, None) == _abi.SOMA_ERR_STATE
    assert _abi.soma_opt_sumsq8(None, None, None, 0, 1.0, None, None) == _abi.SOMA_ERR_STATE


def test_the_fp32_call_does_not_see_scales_of_an_earlier_one():
    """After a refused call with scales, the same handle refuses a list of bytes as fp32 moments by their alignment."""
    opt = SomaOpt(0)
    opt.add_group(lr=1e-3)
    arr = (_abi.soma_tensor_t * 1)(entry(exp_avg=3 * P + 1, group=9))
    sc = (_abi.soma_scales_t * 1)((5 * P, 6 * P))
    assert _abi.soma_opt_step8(opt.handle, arr, sc, 1, 1.0, 1.0, None) == _abi.SOMA_ERR_BAD_GROUP
    arr[0].group = 0
    assert _abi.soma_opt_step(opt.handle, arr, 1, 1.0, 1.0, None) == _abi.SOMA_ERR_ALIGNMENT


def test_the_list_refuses():
    p, g = torch.zeros(600), torch.zeros(600)
    (m, ms), (v, vs) = zeros_8bit(p), zeros_8bit(p)
    assert ms.numel() == 3

    def make(**kw):
        a = dict(params=[p], grads=[g], exp_avgs=[m], exp_avg_sqs=[v], groups=[0], exp_avg_scales=[ms],
                 exp_avg_sq_scales=[vs])
        return TensorList(**{**a, **kw})
    tl = make()
    assert tl.scales[0].exp_avg == ms.data_ptr() and tl.array[0].exp_avg == m.data_ptr()
    for kw, error, word in ((dict(exp_avg_scales=None), ValueError, "go together"),
                            (dict(exp_avg_sq_scales=[None]), ValueError, "go together"),
                            (dict(exp_avg_scales=[ms, ms]), ValueError, "one entry per tensor"),
                            (dict(exp_avg_scales=[ms[:2]]), ValueError, "3 scales expected"),
                            (dict(exp_avg_sq_scales=[vs.double()]), TypeError, "float32"),
                            (dict(exp_avgs=[p]), TypeError, "float8"), (dict(exp_avgs=[m[:599]]), ValueError, "numel"),
                            (dict(exp_avg_scales=[None], exp_avg_sq_scales=[None]), TypeError, "float32"),
                            (dict(exp_avg_scales=None, exp_avg_sq_scales=None), TypeError, "float32")):
        with pytest.raises(error, match=word):
            make(**kw)
    mixed = TensorList([p, p], [g, g], [m, p], [v, p], groups=[0, 0], exp_avg_scales=[ms, None],
                       exp_avg_sq_scales=[vs, None])
    assert mixed.scales[1].exp_avg is None and mixed.array[1].exp_avg == p.data_ptr()
    assert make(trainable=[False]).scales[0].exp_avg is None


def test_conversion_on_the_cpu():
    x = torch.tensor([0.0, 1.0, -2.0, 1e-9])
    codes, scales = to_8bit(x)
    assert codes.dtype == F8 and torch.equal(from_8bit(codes, scales)[:3], x[:3])


def test_a_converted_second_moment_stays_above_0():
    x = torch.cat([torch.tensor([1.0, 1e-6, 0.0, 1e-30]), torch.zeros(252), torch.tensor([0.0, 2.0 ** -60, 1e25, 3.0])])
    codes, scales = to_8bit(x, second_moment=True)
    assert torch.equal(from_8bit(codes, scales) > 0, x > 0)
    # at least the first code, 2^-9, of a block whose largest is 448; what is above it is rounded as any moment is
    assert codes[1].item() == codes[3].item() == 2.0 ** -9
    plain, plain_scales = to_8bit(x)
    above = plain.float() > 0
    assert torch.equal(scales, plain_scales) and torch.equal(codes.float()[above], plain.float()[above])
    nothing = to_8bit(torch.zeros(300), second_moment=True)
    assert not nothing[0].float().any() and not nothing[1].any()


def test_struct_layout():
    assert ctypes.sizeof(_abi.soma_scales_t) == 16 and _abi.SOMA_STATE_BLOCK == 256
