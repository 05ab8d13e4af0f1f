"""What the tensor calls of the 8-bit operators hand to the library, and what they refuse,
without a GPU: CPU tensors that call themselves CUDA tensors, and a library that writes
its arguments down."""
import pytest
import torch

import dense_fp32_gemm_05_gb300 as sg

E4M3 = torch.float8_e4m3fn


class Tensor:
    """A CPU tensor on "device 0"."""

    def __init__(self, t):
        self.t = t

    is_cuda = True
    device = torch.device("cpu")

    def get_device(self):
        return 0

    def __getattr__(self, name):
        return getattr(self.t, name)


@pytest.fixture
def calls(monkeypatch):
    """The library's calls: (entry point, arguments)."""
    made = []

    class Library:
        def __getattr__(self, name):
            def call(*args):
                made.append((name, args))
                return 0
            return call

    monkeypatch.setattr(sg, "load", lambda: Library())
    monkeypatch.setattr(sg, "_current_stream", lambda device: 0)
    monkeypatch.setattr(sg, "_raw_device", lambda: 0, raising=False)
    return made


def _f32(*shape):
    return torch.zeros(shape)


def _codes(*shape):
    return torch.zeros(shape, dtype=torch.uint8).view(E4M3)


def _overlapping(rows, cols, codes=False):
    """Tensors of that shape in which rows share memory."""
    make = _codes if codes else _f32
    flat = make(1, rows + cols)
    return [make(1, cols).expand(rows, cols), flat.as_strided((rows, cols), (1, 1)),
            make(1, rows * cols).as_strided((rows, cols), (cols - 1, 1)),
            make(cols * rows).unfold(0, cols, cols // 2)[:rows].expand(-1, cols)]


def _quantize(**change):
    a = dict(X=_f32(16, 256), Q=_codes(16, 256), S=_f32(2, 16))
    a.update(change)
    return sg.fp8_quantize(Tensor(a["X"]), Q=Tensor(a["Q"]), S=Tensor(a["S"]))


def _product(**change):
    a = dict(A=_codes(16, 256), SA=_f32(2, 16), B=_codes(40, 256), SB=_f32(2, 40), C=_f32(16, 40))
    a.update(change)
    return sg.fp8_gemm(*(Tensor(a[n]) for n in ("A", "SA", "B", "SB", "C")), b_group=1)


def _moe(**change):
    T, D, F, E, k = 6, 128, 64, 4, 2
    a = dict(x=_f32(T, D), router=_f32(E, D), gate=_codes(E, F, D), s_gate=_f32(E, 1, 1), up=_codes(E, F, D),
             s_up=_f32(E, 1, 1), down=_codes(E, D, F), s_down=_f32(E, 1, 1), y=_f32(T, D), logits=_f32(T, E),
             indices=torch.zeros((T, k), dtype=torch.int32), weights=_f32(T, k))
    a.update(change)
    a = {n: Tensor(t) for n, t in a.items()}
    return sg.moe(topk=k, **a)


@pytest.mark.parametrize("run,name,rows,cols,codes", [
    (_quantize, "X", 16, 256, False), (_quantize, "Q", 16, 256, True), (_quantize, "S", 2, 16, False),
    (_product, "A", 16, 256, True), (_product, "SA", 2, 16, False), (_product, "B", 40, 256, True),
    (_product, "SB", 2, 40, False), (_product, "C", 16, 40, False), (_moe, "x", 6, 128, False),
    (_moe, "y", 6, 128, False)])
def test_rows_that_overlap_are_refused(calls, run, name, rows, cols, codes):
    for t in _overlapping(rows, cols, codes):
        assert t.shape == (rows, cols) and t.stride(0) < cols
        with pytest.raises(ValueError, match="overlap"):
            run(**{name: t})
    assert not calls


def test_leading_dimensions(calls):
    """Packed and padded rows as they are; a single row's stride, and an empty tensor's, mean nothing."""
    X, Q, S = _f32(16, 300)[:, :256], _codes(16, 272)[:, :256], _f32(2, 20)[:, :16]
    _quantize(X=X, Q=Q, S=S)
    name, args = calls.pop()
    assert name == "sgemm_fp8_quantize"
    assert args[:5] == (16, 256, X.data_ptr(), sg.TYPE_F32, 300) and args[7:12] == (Q.data_ptr(), sg.TYPE_E4M3, 272,
                                                                                    S.data_ptr(), 20)
    for one in (_f32(1, 256), _f32(1, 256).expand(7, 256)[3:4], _f32(9, 999)[:1, :256], _f32(1, 300).as_strided((1, 256), (0, 1))):
        _quantize(X=one, Q=_codes(1, 256), S=_f32(2, 1))
        assert calls.pop()[1][4] == 256
    _quantize(X=_f32(16, 1).as_strided((16, 1), (1, 7)), Q=_codes(16, 1), S=_f32(1, 16))
    assert calls.pop()[1][4] == 1
    _quantize(X=_f32(0, 256), Q=_codes(0, 256), S=_f32(2, 0))
    assert calls.pop()[1][4] == 256
    _quantize(X=_f32(16, 0), Q=_codes(16, 0), S=_f32(0, 16))
    assert calls.pop()[1][4] == 1
    _product(A=_codes(16, 512)[:, 128:384], C=_f32(16, 41)[:, :40])
    args = calls.pop()[1]
    assert args[8] == 512 and args[-2] == 41


@pytest.mark.parametrize("run", [_quantize, _product, _moe])
def test_tensors_of_another_device_than_the_current_one_are_refused(calls, run, monkeypatch):
    run()
    assert len(calls) == 1
    monkeypatch.setattr(sg, "_raw_device", lambda: 1, raising=False)
    with pytest.raises(ValueError, match="device"):
        run()
    assert len(calls) == 1
