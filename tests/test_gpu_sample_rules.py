"""sample() where a rule of include/fq.h decides alone, by hand."""
import pytest
import torch

import fp8_quant_memory_gb300 as fq

pytestmark = pytest.mark.gpu


@pytest.fixture(autouse=True)
def _device_state(cuda_ok):
    yield
    torch.cuda.synchronize()
    assert fq.device_status(clear=True) == 0


@pytest.mark.parametrize("dt", [torch.bfloat16, torch.float16])
@pytest.mark.parametrize("V", [7, 1000, 70001])
@pytest.mark.parametrize("cuts", ["min_p", "top_p", "top_k", "long top_k"])
@pytest.mark.parametrize("min_p", [1.0, 1.5, 3e38, float("inf")])
def test_min_p_above_one_counts_as_one(min_p, cuts, V, dt):
    """Four equal largest values (of 7 tokens: two) stay, whatever other cuts leave them all: u picks among them alike."""
    at = [1, 5] if V == 7 else [3, V // 3, V // 2, V - 1]
    x = torch.linspace(-3.0, 1.0, V).repeat(len(at), 1)
    x[:, at] = 2.0
    u = torch.tensor([(i + 0.5) / len(at) for i in range(len(at))])
    full = lambda v, t=torch.float32: torch.full((len(at),), v, dtype=t, device="cuda")
    more = {"top_p": dict(top_p=full(0.9999)), "top_k": dict(top_k=full(5, torch.int32)), "long top_k": dict(top_k=full(900, torch.int32))}
    token, logprob = fq.sample(x.to(dt).cuda(), u.cuda(), min_p=full(min_p), want_logprob=True, **more.get(cuts, {}))
    assert token.tolist() == at
    assert bool(((logprob.cpu().double() + torch.tensor(float(len(at))).double().log()).abs() <= 2.0 ** -21).all())
