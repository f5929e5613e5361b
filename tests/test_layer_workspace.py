"""The workspace of qr_gemm_i8, as include/qr_layer.h has it: no size needs one, NULL will do, and a buffer that is passed
all the same is neither read nor written."""
import pytest
import torch


def test_no_size_needs_a_workspace():
    from quantized_two_stage_amd import qr
    for M in (0, 1, 8, 9, 333, 8192, 1 << 22):
        for N in (1, 64, 5003, 1 << 22):
            for K in (1, 2050, 131071):
                assert qr.qr_gemm_i8_workspace_bytes(M, N, K) == 0
    assert qr.alloc_gemm_workspace(333, 5003, 2050) is None


@pytest.mark.gpu
@pytest.mark.parametrize("M,N,K", [(1, 300, 8192), (9, 77, 1000), (48, 4200, 4096), (333, 2001, 4096), (1024, 1024, 512)])
def test_a_workspace_is_left_alone(M, N, K):
    from quantized_two_stage_amd import qr
    g = torch.Generator(device="cuda").manual_seed(M)
    (a, sa), (b, sb) = qr.alloc_q8(M, K), qr.alloc_q8(N, K)
    for codes, scales in ((a, sa), (b, sb)):
        codes.copy_(torch.randint(-128, 128, codes.shape, generator=g, device="cuda", dtype=torch.int8))
        scales.copy_(torch.rand(scales.shape, generator=g, device="cuda") * 0.01)
    outs = []
    for fill in (None, 0, 0xA7):
        # not aligned, and of no particular size: the call has no use for it
        whole = None if fill is None else torch.full((4097,), fill, dtype=torch.uint8, device="cuda")
        c = torch.empty(M, N, dtype=torch.bfloat16, device="cuda")
        qr.qr_gemm_i8(a, sa, b, sb, c, workspace=None if whole is None else whole[1:])
        torch.cuda.synchronize()
        assert whole is None or bool((whole == fill).all())
        outs.append(c.view(torch.int16))
    assert torch.equal(outs[0], outs[1]) and torch.equal(outs[0], outs[2])
