"""GPU: the codes of msa_add_rms_norm_fp8 where the norm itself is exact."""
import pytest
import torch

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def msa():
    if not torch.cuda.is_available():
        pytest.skip("needs a GPU")
    import __graft_entry__
    __graft_entry__.build()
    import block_sparse_attention_05_gb300 as m
    torch.cuda.set_device(0)
    return m


def _bf16(bits):
    return torch.tensor(bits, dtype=torch.int32).to(torch.int16).view(torch.bfloat16)


@pytest.mark.parametrize("top", [1.0, 1.25, 1.375, 1.9921875, 3.0, 4.15625, 5.0, 7.0, 3.0 * 2.0 ** 90, 5.0 * 2.0 ** -90])
@pytest.mark.parametrize("pad", [0, 3])
def test_codes_are_those_of_the_quotient(msa, top, pad):
    """Rows of +-1: the mean of their squares is 1, y = +-(1 / sqrt(1 + eps)) gamma with IEEE operations, and the quotient of
    two gammas comes to a midpoint between two codes now and then.  gamma: every bf16 value from 2^-20 of the largest up."""
    every = _bf16(list(range(0x0080, 0x7F80)))
    gamma = every[(every.float() <= top) & (every.float() >= top * 2.0 ** -20)]
    gamma = torch.cat([gamma, torch.full((pad,), top, dtype=torch.bfloat16)])
    width = gamma.numel()
    x = torch.where(torch.arange(width) % 3 == 0, -1.0, 1.0).to(torch.bfloat16)[None].repeat(5, 1)
    one, gamma_gpu, x_gpu = torch.tensor(1.0), gamma.cuda(), x.cuda()
    for k in range(40):
        eps = torch.tensor(k * 0.0371)
        y = x.float() * (one / torch.sqrt(one + eps)) * gamma.float()
        scale = y.abs().max() / torch.tensor(448.0)
        total, codes, got = msa.msa_add_rms_norm_fp8(x_gpu, gamma_gpu, eps=float(eps))
        assert torch.equal(total, x_gpu) and (got.cpu() == scale).all()
        assert torch.equal(codes.cpu(), (y / scale).to(torch.float8_e4m3fn).view(torch.uint8)), k
