"""Calls around the experts and on int4 weights take tensors of the current device alone: each
operand, workspace, scratch and packed weights.  On the host: tensors that claim a device, and a
library that is not called."""

import pytest
import torch

from grouped_ffn_gb300 import moe as m

BF, F32, I32, U8 = torch.bfloat16, torch.float32, torch.int32, torch.uint8


class On(torch.Tensor):
    """A host tensor that says it is on a CUDA device."""
    dev = 0
    is_cuda = property(lambda self: self.dev >= 0)
    __torch_function__ = torch._C._disabled_torch_function_impl

    def get_device(self):
        return self.dev


def on(*shape, t=BF, dev=0):
    x = torch.zeros(*shape, dtype=t).as_subclass(On)
    x.dev = dev
    return x


class Library:
    def __init__(self):
        self.calls = 0

    def __getattr__(self, name):
        def call(*a):
            self.calls += 1
            return 256 if name.endswith("bytes") else 0
        return call


T, H, k, n = 3, 64, 2, 8
CFG = m.BlockCfg()


def operands():
    row, rows, w = lambda: on(T, H), lambda: on(n, H), lambda: on(T, k, t=F32)
    dest, ws, scratch, h = on(T, k, t=I32), on(256, t=U8), on(4096, t=U8), lambda: on(H, t=F32)
    token = lambda: on(T, t=F32)
    return dict(
        moe_norm=(dict(x=row(), weight=h(), out=row()), dict(eps=1e-6)),
        moe_combine_norm=(dict(y_perm=rows(), dest_row=dest, topk_w=w(), residual=row(), y=row(), ws=ws, shared=row(),
                               weight=h(), gate=token(), next_weight=h(), next_out=row()), dict(cfg=CFG)),
        moe_combine_backward=(dict(grad_y=row(), y_perm=rows(), dest_row=dest, topk_w=w(), grad_y_perm=rows(),
                                   grad_topk_w=w(), ws=ws), {}),
        moe_permute_backward=(dict(grad=rows(), dest_row=dest, grad_x=row(), ws=ws, add=row()), {}),
        moe_combine_norm_backward=(dict(grad_y=row(), y_perm=rows(), dest_row=dest, topk_w=w(), grad_y_perm=rows(),
                                        grad_topk_w=w(), ws=ws, scratch=scratch, shared=row(), weight=h(),
                                        gate=token(), grad_shared=row(), grad_weight=h(), grad_gate=token()),
                                   dict(cfg=CFG)),
        moe_norm_backward=(dict(grad=rows(), x=row(), weight=h(), grad_x=row(), grad_weight=h(), ws=ws,
                                scratch=scratch, dest_row=dest, add=row(), residual_grad=row()), dict(eps=1e-6)),
        moe_grouped_product_int4=(dict(x=on(n, 32), seg_offsets=on(3, t=I32), seg_expert=on(2, t=I32),
                                       w=on(512, t=U8), out=on(n, 8), ws=ws), {}),
        pack_weights_int4=(dict(codes=on(2, 8, 16, t=U8), scales=on(2, 8, 1), zeros=on(2, 8, 1, t=U8)),
                           dict(epilogue=m.MOE_EPI_NONE)),
    )


CALLS = [(name, arg) for name, (tensors, _) in operands().items() for arg in (None, *tensors)]


@pytest.mark.parametrize("name,arg", CALLS)
def test_a_tensor_of_another_device(monkeypatch, name, arg):
    library = Library()
    monkeypatch.setattr(m, "lib", lambda: library)
    monkeypatch.setattr(m, "_devices", 2)
    monkeypatch.setattr(torch._C, "_cuda_getCurrentRawStream", lambda dev: 0, raising=False)
    monkeypatch.setattr(torch._C, "_cuda_getDevice", lambda: 0, raising=False)
    tensors, rest = operands()[name]

    def run():
        t = dict(tensors)
        if name == "moe_grouped_product_int4":
            t["w"] = m.Int4Weights(t["w"], 2, 8, 32, 32, False, m.MOE_EPI_NONE)
        return getattr(m, name)(**t, **rest)

    if arg is None:
        run()
        assert library.calls
        return
    for dev, error in ((1, ValueError), (-1, TypeError)):
        tensors[arg].dev = dev
        with pytest.raises(error, match="device" if dev == 1 else "CUDA"):
            run()
    assert not library.calls
