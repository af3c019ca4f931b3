"""Stream arguments by handle, and what is read on streams other than their own."""
import pytest
import torch

import fsdp_sharded_mixed_flatparameter_gb300 as pkg
from fsdp_sharded_mixed_flatparameter_gb300.optimizer import torch_stream

pytestmark = pytest.mark.gpu


def gen(seed):
    return torch.Generator().manual_seed(seed)


def test_handle_0_is_the_default_stream():
    dev = torch.device("cuda", torch.cuda.current_device())
    assert torch_stream(0, dev) == torch.cuda.default_stream(dev)
    s = torch.cuda.Stream()
    assert torch_stream(s.cuda_stream, dev).cuda_stream == s.cuda_stream
    with torch.cuda.stream(s):
        assert torch_stream(None, dev) == s and torch_stream(0, dev) == torch.cuda.default_stream(dev)


def test_a_step_on_handle_0_waits_for_its_own_norm():
    # the norm is read on the stream that computes it, behind a pause there
    n = 3000
    opt = pkg.FlatShardAdamW([n], lr=1e-2, device="cuda")
    g = torch.randn(n, generator=gen(1)).cuda()
    want = opt.step_tensors([g]).norm
    opt.device_table([h := g * 2])
    torch.cuda.synchronize()
    torch.cuda._sleep(200_000_000)
    assert opt.step_tensors([h], stream=0).norm == 2 * want and opt.t == 2
