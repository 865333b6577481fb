"""Gradients that go to an asynchronous anchor update and, clipped in place, to the step behind it: the anchor
momentum is that of the gradients as they were given."""
import pytest
import torch

from tests.gpu_harness import say
from tests.test_gpu_train import gen, randn, sco

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("shapes,rounds", [([(96, 64)], 4), ([(1024, 512)] * 24 + [(320, 1024)], 3)])
@pytest.mark.parametrize("by_hand", [False, True])
def test_step_clips_after_the_anchor_has_read(shapes, rounds, by_hand, dtype):
    say(f"case: anchor read {len(shapes)} matrices by hand {by_hand} {dtype}")
    m = sco()
    runs = []
    for shared in (True, False):
        g = gen(81)
        opt = m.SpectralAdamW(shapes, g_dtype=dtype, device=torch.device("cuda", 0))
        W = [randn(g, *s) for s in shapes]
        kept = []
        for _ in range(rounds):
            G = [randn(g, *s, dtype=dtype) for s in shapes]
            anchor = G if shared else [x.clone() for x in G]
            torch.cuda.synchronize()  # nothing queued that would keep the clip behind the update
            opt.anchor_update_async(anchor)
            if by_hand:
                opt.anchor_read_wait()
                norm = m.clip_grads(G, 1e-3).norm
                opt.step(W, G)
            else:
                norm = opt.step(W, G, max_norm=1e-3).norm
            opt.refresh_wait()
            kept += [norm, *G]
        kept += [opt.get_state(i, "m_anc") for i in range(len(shapes))]
        torch.cuda.synchronize()
        runs.append([x.clone() for x in kept + W])
        opt.close()
    for a, b in zip(*runs):
        assert torch.equal(a, b)


def test_read_wait_without_an_update():
    """Nothing pending: never asked for, completed, and on another stream than the update's."""
    m, g = sco(), gen(82)
    opt = m.SpectralAdamW([(64, 96)], device=torch.device("cuda", 0))
    G, W = [randn(g, 64, 96)], [randn(g, 64, 96)]
    opt.anchor_read_wait()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    opt.anchor_update_async(G)
    with torch.cuda.stream(side):
        opt.anchor_read_wait()
        G[0].zero_()
    opt.refresh_wait()
    opt.anchor_read_wait()
    torch.cuda.current_stream().wait_stream(side)
    opt.step(W, G, max_norm=1.0)
    assert torch.count_nonzero(opt.get_state(0, "m_anc")) == 64 * 96
    opt.close()


def test_a_closed_optimizer_leaves_the_gradients():
    """step refuses before it scales anything."""
    m, g = sco(), gen(83)
    opt = m.SpectralAdamW([(64, 96)], device=torch.device("cuda", 0))
    G, W = [randn(g, 64, 96)], [randn(g, 64, 96)]
    before = G[0].clone()
    opt.close()
    with pytest.raises(m.ScoptError):
        opt.step(W, G, max_norm=1e-3)
    assert torch.equal(G[0], before)
