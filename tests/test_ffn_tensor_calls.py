"""What the tensor calls of the feed-forward and 4-bit operators hand to the library, and what
they refuse, without a GPU: CPU tensors that call themselves CUDA tensors, and a library that
writes its arguments down."""
import pytest
import torch

import dense_fp32_gemm_05_gb300 as sg
from tests.test_fp8_tensor_calls import Tensor, calls  # noqa: F401  (a fixture)

BF16, E4M3 = torch.bfloat16, torch.float8_e4m3fn
T, D, F = 6, 40, 264


def _bf16(*shape):
    return torch.zeros(shape, dtype=BF16)


def _u8(*shape):
    return torch.zeros(shape, dtype=torch.uint8)


def _ffn(kept=(), **change):
    a = dict(x=_bf16(T, D), gate=_bf16(F, D), up=_bf16(F, D), down=_bf16(D, F), y=_bf16(T, D), h=_bf16(T, F))
    a.update(change)
    more = {"kept": tuple(Tensor(t) for t in kept)} if kept else {}
    return sg.ffn(**{n: Tensor(t) if isinstance(t, torch.Tensor) else t for n, t in a.items()}, **more)


def _codes():
    return (_u8(T, F).view(E4M3), _u8(T, F).view(E4M3), _bf16(3, T), _bf16(3, T))


def _backward(kept=None, scratch=None, **change):
    a = dict(dy=_bf16(T, D), x=_bf16(T, D), gate=_bf16(F, D), up=_bf16(F, D), down=_bf16(D, F), dx=_bf16(T, D),
             dgate=_bf16(F, D), dup=_bf16(F, D), ddown=_bf16(D, F))
    a.update(change)
    kept = _codes() if kept is None else kept
    scratch = [_bf16(T, F) for _ in range(3)] if scratch is None else scratch
    return sg.ffn_backward(**{n: Tensor(t) if isinstance(t, torch.Tensor) else t for n, t in a.items()},
                           kept=tuple(Tensor(t) for t in kept), scratch=tuple(Tensor(t) for t in scratch))


def _quantize(symmetric=False, **change):
    a = dict(W=torch.zeros(10, 70), Q=_u8(10, 35), S=torch.zeros(3, 10), Z=_u8(3, 10), V=_bf16(10, 70))
    a.update(change)
    return sg.q4_quantize(**{n: t if t is None else Tensor(t) for n, t in a.items()}, group=32, symmetric=symmetric)


def _q4(group=32, activation=None, **change):
    a = dict(X=_bf16(3, 70), Q=_u8(10, 48)[:, :35], S=torch.zeros(3, 10), C=torch.zeros(3, 10), Z=_u8(3, 10),
             Q2=_u8(10, 48)[:, :35], S2=torch.zeros(3, 10), Z2=_u8(3, 10))
    a.update(change)
    return sg.q4_gemm(**{n: t if t is None else Tensor(t) for n, t in a.items()}, group=group, activation=activation)


def test_what_the_library_gets(calls):
    _ffn()
    name, args = calls.pop()
    assert name == "sgemm_ffn" and args[:3] == (T, D, F) and args[10:18] == (sg.ACT_SILU, sg.TYPE_BF16, None, None, F, None, None, 1)
    x = _bf16(T, 48)[:, :D]
    _ffn(_codes(), x=x, activation=sg.ACT_GELU)
    args = calls.pop()[1]
    assert args[3:5] == (x.data_ptr(), 48) and args[10:12] == (sg.ACT_GELU, sg.TYPE_E4M3) and args[14] == F and args[17] == T
    _ffn((_bf16(T, 300)[:, :F], _bf16(T, 300)[:, :F]))
    args = calls.pop()[1]
    assert args[11] == sg.TYPE_BF16 and args[14] == 300 and args[15:18] == (None, None, 1)
    _backward(accumulate=True)
    name, args = calls.pop()
    assert name == "sgemm_ffn_backward" and args[:3] == (T, D, F) and args[26:28] == (sg.TYPE_BF16, 1) and args[19] == T
    _backward(dgate=torch.zeros(F, 44)[:, :D], dup=torch.zeros(F, 44)[:, :D], ddown=torch.zeros(D, F))
    args = calls.pop()[1]
    assert args[26] == sg.TYPE_F32 and args[30] == 44 and args[32] == F
    _quantize()
    name, args = calls.pop()
    assert name == "sgemm_q4_quantize" and args[:2] == (10, 70) and args[5] == 32 and args[7] == 35 and args[10] == 10
    assert args[12:14] == (sg.TYPE_BF16, 70)
    _quantize(True, Z=None, V=None)
    args = calls.pop()[1]
    assert args[9] is None and args[11] is None
    _q4()
    name, args = calls.pop()
    assert name == "sgemm_q4" and args[:3] == (3, 10, 70) and args[12:16] == (48, 10, 32, sg.ACT_SILU)
    _q4(Q2=None, S2=None, Z2=None)
    args = calls.pop()[1]
    assert args[9:12] == (None, None, None) and args[15] == sg.ACT_NONE


F32 = torch.zeros


@pytest.mark.parametrize("run,change", [
    (_ffn, dict(x=F32(T, D))), (_ffn, dict(x=_bf16(T, D, 1))), (_ffn, dict(gate=_bf16(F, D + 1))), (_ffn, dict(gate=_bf16(F))),
    (_ffn, dict(up=_bf16(F + 1, D))), (_ffn, dict(up=_bf16(F, 48)[:, :D])), (_ffn, dict(down=_bf16(F, D))), (_ffn, dict(y=_bf16(T, F))),
    (_ffn, dict(h=F32(T, F))), (_ffn, dict(x=_bf16(D, T).t())), (_ffn, dict(kept=(_bf16(T, F),))), (_ffn, dict(kept=_codes()[:2])),
    (_ffn, dict(kept=_codes()[:3])), (_ffn, dict(kept=(_bf16(T, F), _bf16(T, F)) + _codes()[2:])),
    (_ffn, dict(kept=(_bf16(T, F), _bf16(T, 300)[:, :F]))), (_ffn, dict(kept=_codes()[:2] + (F32(3, T), F32(3, T)))),
    (_ffn, dict(kept=_codes()[:2] + (_bf16(2, T), _bf16(2, T)))), (_ffn, dict(keep=torch.float16)),
    (_ffn, dict(kept=_codes(), keep=BF16)), (_ffn, dict(x=_bf16(1, D).expand(T, D))),
    (_backward, dict(dy=_bf16(T, D + 8))), (_backward, dict(dgate=F32(F, D))), (_backward, dict(dup=_bf16(F, 48)[:, :D])),
    (_backward, dict(ddown=F32(D, F))), (_backward, dict(dx=F32(T, D))), (_backward, dict(scratch=[_bf16(T, F)] * 2)),
    (_backward, dict(scratch=[_bf16(T, F), _bf16(T, F), _bf16(T, 272)[:, :F]])), (_backward, dict(kept=(_bf16(T, F), _bf16(T, F - 1)))),
    (_quantize, dict(W=_u8(10, 70))), (_quantize, dict(Q=_u8(10, 36))), (_quantize, dict(Q=F32(10, 35))), (_quantize, dict(S=F32(3, 11))),
    (_quantize, dict(Z=_u8(2, 10))), (_quantize, dict(Z=_u8(3, 12)[:, :10])), (_quantize, dict(V=F32(10, 71))),
    (_quantize, dict(symmetric=True)), (_quantize, dict(Q=_u8(1, 35).expand(10, 35))),
    (_q4, dict(X=_u8(3, 70))), (_q4, dict(group=16)), (_q4, dict(group=64)), (_q4, dict(Q=_u8(10, 36))), (_q4, dict(S=F32(3, 9))),
    (_q4, dict(Z=None)), (_q4, dict(Z2=None)), (_q4, dict(Q2=_u8(10, 64)[:, :35])), (_q4, dict(S2=F32(3, 12)[:, :10])),
    (_q4, dict(Q2=None)), (_q4, dict(Q2=None, S2=None)), (_q4, dict(C=F32(3, 11))), (_q4, dict(C=_u8(3, 10)))])
def test_refusals(calls, run, change):
    with pytest.raises(ValueError):
        run(**change)
    assert not calls


def test_accumulating_needs_gradients(calls):
    x, w, d = _bf16(T, D), _bf16(F, D), _bf16(D, F)
    with pytest.raises(ValueError, match="accumulate"):
        sg.ffn_backward(*(Tensor(t) for t in (x, x, w, w, d)), tuple(Tensor(t) for t in _codes()), dgate=Tensor(w), dup=Tensor(w),
                        accumulate=True)
    assert not calls


@pytest.mark.parametrize("run", [_ffn, _backward, _quantize, _q4])
def test_tensors_of_another_device_than_the_current_one_are_refused(calls, run, monkeypatch):
    run()
    assert len(calls) == 1
    monkeypatch.setattr(sg, "_raw_device", lambda: 1, raising=False)
    with pytest.raises(ValueError, match="device"):
        run()
    assert len(calls) == 1
