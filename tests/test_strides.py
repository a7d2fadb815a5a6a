"""CPU-only checks of how the operators with allocated results read a tensor's layout. The tensors
say that they live on a GPU, so that every check before the launch runs; each of these calls has to
end in such a check."""
import pytest
import torch

import dense_fp32_matrix_08_gb300 as sg


class OnGpu(torch.Tensor):
    is_cuda = True


def on_gpu(t):
    return t.as_subclass(OnGpu)


def overlapping(rows, cols, dtype=torch.float32):
    """Views whose rows share elements: one row for all, and a window that slides by one."""
    bytes_ = torch.zeros(rows + cols, dtype=torch.uint8) if dtype.itemsize == 1 else None
    flat = bytes_.view(dtype) if bytes_ is not None else torch.zeros(rows + cols, dtype=dtype)
    return [on_gpu(flat[:cols].as_strided((rows, cols), (0, 1))),
            on_gpu(flat.as_strided((rows, cols), (1, 1)))]


@pytest.mark.parametrize("which", [0, 1])
@pytest.mark.parametrize("cols", [2, 128, 300])
def test_quantize_refuses_overlapping_rows(which, cols):
    x = overlapping(8, cols)[which]
    for call in (sg.f8_quantize, sg.f8_quantize_pair):
        with pytest.raises(ValueError, match="overlap"):
            call(x)
    with pytest.raises(ValueError, match="overlap"):
        sg.f8_quantize(x, (128, 128))


@pytest.mark.parametrize("which", [0, 1])
def test_matmul_refuses_overlapping_rows(which):
    q = on_gpu(torch.zeros(32, 160, dtype=torch.uint8).view(torch.float8_e4m3fn))
    s, w = on_gpu(torch.ones(32, 2)), on_gpu(torch.ones(1, 2))
    bad = overlapping(32, 160, torch.float8_e4m3fn)[which]
    with pytest.raises(ValueError, match="a's rows overlap"):
        sg.f8_matmul(bad, s, q, w, transb=True)
    with pytest.raises(ValueError, match="b's rows overlap"):
        sg.f8_matmul(q, s, bad, w, transb=True)
    for dtype in (torch.float32, torch.bfloat16):
        with pytest.raises(ValueError, match="out's rows overlap"):
            sg.f8_matmul(q, s, q, w, transb=True, out=overlapping(32, 32, dtype)[which])


@pytest.mark.parametrize("which", [0, 1])
def test_orthogonalize_refuses_overlapping_rows(which):
    g = on_gpu(torch.zeros(6, 9))
    bad = overlapping(6, 9)[which]
    with pytest.raises(ValueError, match="g's rows overlap"):
        sg.orthogonalize(bad)
    with pytest.raises(ValueError, match="g's rows overlap"):
        sg.orthogonalize(bad[None].expand(2, 6, 9))
    with pytest.raises(ValueError, match="out's rows overlap"):
        sg.orthogonalize(g, out=bad)


def test_one_row_or_column_needs_no_stride():
    """The stride of a dimension of one element says nothing; two rows of one column still need one."""
    from dense_fp32_matrix_08_gb300 import f8, newton_schulz
    flat = torch.zeros(400)
    for shape, strides, ld in (((1, 7), (0, 1), 7), ((1, 7), (3, 1), 7), ((5, 1), (1, 9), 1),
                               ((5, 1), (4, 1), 4), ((5, 3), (3, 1), 3), ((5, 0), (1, 1), 1),
                               ((0, 4), (4, 1), 4)):
        t = on_gpu(flat.as_strided(shape, strides))
        assert f8._rows("x", t) == (*shape, ld)
        assert newton_schulz._matrices("x", t)[1] == ld
    for helper in (f8._rows, newton_schulz._matrices):
        with pytest.raises(ValueError, match="overlap"):
            helper("x", on_gpu(flat.as_strided((5, 1), (0, 1))))


@pytest.mark.parametrize("dtype", [torch.float32, torch.float8_e4m3fn])
def test_sizes_past_32_bits_are_refused(dtype):
    """Sizes reach the library as 32-bit integers: one that does not fit must not become another one."""
    from dense_fp32_matrix_08_gb300 import f8, newton_schulz
    far = on_gpu(torch.empty((2, (1 << 32) + 16), dtype=dtype, device="meta"))
    for t in (far, far[:, :6], far.t()[:1 << 31].t(), far.reshape(-1, 1)):
        with pytest.raises(ValueError, match="2\\^31"):
            f8._rows("x", t)
        if dtype is torch.float32:
            with pytest.raises(ValueError, match="2\\^31"):
                newton_schulz._matrices("x", t)
    if dtype is torch.float32:
        for call in (sg.f8_quantize, sg.f8_quantize_pair, sg.orthogonalize):
            with pytest.raises(ValueError, match="2\\^31"):
                call(far[:, :6])
        with pytest.raises(ValueError, match="2\\^31"):
            sg.orthogonalize(on_gpu(torch.empty(((1 << 32) + 1, 2, 2), device="meta")))


def test_steps_past_32_bits_are_refused(monkeypatch):
    monkeypatch.setattr(torch._C, "_cuda_getDevice", lambda: 0, raising=False)
    monkeypatch.setattr(torch._C, "_cuda_getCurrentRawStream", lambda device: 0, raising=False)
    g = on_gpu(torch.empty((0, 4)))
    assert sg.orthogonalize(g, steps=64, out=g) is g
    for steps in (65, (1 << 32) + 5, -1, -(1 << 32)):
        with pytest.raises(sg.SgemmError) as e:
            sg.orthogonalize(g, steps=steps, out=g)
        assert e.value.status == -8
