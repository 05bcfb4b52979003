"""The operators around the path at the ends of their ranges: more tokens than
one launch has threads for, and than an int32 counts."""
import pytest
import torch

from tests import ops_ref as ref
from tests.gpu_util import say

pytestmark = pytest.mark.gpu
BF, F32 = torch.bfloat16, torch.float32


@pytest.fixture(scope="module")
def cco():
    import combine_symmetric_memory_amd as m
    assert torch.cuda.is_available()
    return m


def test_more_tokens_than_a_launch_has_threads(cco):
    # 64 lanes a token: from 2^26 tokens on one launch would need 2^32 threads
    T, E = 2 ** 26 + 77, 2
    say("case: route T=%d" % T)
    g = torch.Generator(device="cuda").manual_seed(1)
    logits = torch.randint(-2, 3, (T, E), generator=g, device="cuda", dtype=torch.int8).to(BF)
    idx, w = cco.route(logits, 1, renorm=True)
    assert torch.equal(idx[:, 0] == 1, logits[:, 1] > logits[:, 0])  # equal: the lower id
    assert bool((w == 1.0).all())
    del w
    dw = torch.ones((T, 1), device="cuda")
    got = cco.route_grad(logits, idx, dw, score="sigmoid")
    # five distinct logits: sigmoid' of the chosen one, 0 for the other
    chosen = torch.gather(logits, 1, idx.long()).double()
    s = torch.sigmoid(chosen)
    want = s * (1 - s)
    # exp and two quotients in 32 bits, rounded once to bf16
    bound = want * (ref.half_step(BF) + 32 * ref.U)
    assert bool(((torch.gather(got, 1, idx.long()).double() - want).abs() <= bound).all())
    assert not bool(torch.gather(got, 1, 1 - idx.long()).any())


def test_tokens_past_the_counts_type_are_refused(cco):
    # 2^32 + 5 rows are not 5 rows
    x = torch.empty((2 ** 32 + 5, 1), dtype=BF, device="cuda")
    with pytest.raises(ValueError):
        cco.route(x, 1)
    with pytest.raises(ValueError):
        cco.block_norm(x, pre=torch.ones(1, device="cuda"))
