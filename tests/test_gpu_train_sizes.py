"""GPU tests of the training-step operators at sizes that their other tests do not reach: the
launch limits of the embedding gradient."""
import pytest
import torch

from tests.gpu_harness import say

pytestmark = pytest.mark.gpu

F64 = torch.float64


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")


def sco():
    import spectral_correction_optimizer_amd as m
    return m


def gen(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    return g


def test_embed_grad_more_crossings_than_a_launch_holds():
    """Over 2^24 stretches of sorted tokens, and every table row crosses thousands of them: more
    crossings than workgroups of 256 threads fit in one launch.  Small integers: every sum is exact."""
    T, V = (1 << 29) + 12345, 4099
    say(f"case: embed_grad T {T} V {V} H 1")
    dy = torch.randint(-8, 8, (T, 1), generator=gen(1), device="cuda", dtype=torch.int8).float()
    ids = torch.arange(T, device="cuda") % V
    dW = sco().embed_grad(dy, ids, V)
    n = T // V
    ref = dy[:n * V].view(n, V).sum(0, dtype=F64)
    ref[:T - n * V] += dy[n * V:, 0]
    assert torch.equal(dW[:, 0].to(F64), ref)
