"""Memory that calls allocate, on a stream of the caller."""

import pytest
import torch


@pytest.mark.gpu
def test_packed_weights_belong_to_the_stream_that_writes_them():
    """A tensor freed while a copy of it is still queued on the current stream: packing on another
    stream does not write into its memory."""
    from grouped_ffn_gb300 import build, moe as m
    build.build()
    E, N, K = 4, 512, 2048
    gen = torch.Generator(device="cuda")
    gen.manual_seed(1)
    codes = torch.randint(0, 256, (E, N, K // 2), generator=gen, device="cuda").to(torch.uint8)
    sf = torch.full((E, N, m.moe_fp4_scale_ld(K, m.MOE_FP4_NV)), 0x38, dtype=torch.uint8, device="cuda")
    want = m.pack_weights_fp4(codes, sf, m.MOE_FP4_NV, m.MOE_EPI_NONE)
    a = torch.randn(4096, 4096, device="cuda")
    held = torch.full_like(want.data, 77)
    copy = torch.empty_like(held)
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    for _ in range(20):
        a = a @ a * 1e-3
    copy.copy_(held)
    del held
    got = m.pack_weights_fp4(codes, sf, m.MOE_FP4_NV, m.MOE_EPI_NONE, side)
    side.synchronize()
    assert torch.equal(got.data, want.data)
    torch.cuda.synchronize()
    assert (copy == 77).all()


@pytest.mark.gpu
def test_a_workspace_belongs_to_the_stream_that_clears_it():
    from grouped_ffn_gb300 import build, moe as m
    build.build()
    a = torch.randn(4096, 4096, device="cuda")
    held = torch.full_like(m.new_workspace(4096, 8, 256), 77)
    copy = torch.empty_like(held)
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    for _ in range(20):
        a = a @ a * 1e-3
    copy.copy_(held)
    del held
    ws = m.new_workspace(4096, 8, 256, stream=side)
    side.synchronize()
    assert not ws.any()
    torch.cuda.synchronize()
    assert (copy == 77).all()
