"""The attention layer where scores, weights and references lie far apart,
against dense 64-bit forms (bounds as derived in attention_ref)."""
import pytest
import torch

from test_gpu_attention import Batch

pytestmark = pytest.mark.gpu


# few query tiles (an item's key tiles are shared out between two pipelines and joined), or many
@pytest.mark.parametrize("heads", [(2, 1), (40, 20)])
@pytest.mark.parametrize("keys", [(200, 300), (100, 400), (300, 400), (300, 301), (130, 260)])
@pytest.mark.parametrize("score", [80.0, 87.0, 87.5, 88.0, 88.5, 91.0, 95.0])
def test_late_scores_in_two_tiles(cpt, cuda_device, score, keys, heads):
    """Two late keys score the same, 80 to 95 above all others, in one tile or in tiles that two
    pipelines take: both weigh as much, whatever reference each pipeline has. A score here is one product of two
    bf16 values, so it is exact; weights, lse and the gradients are checked within the usual bounds."""
    b = Batch(cpt, 0, 1, [512], *heads, 64, 512, 0, scale=1.0)
    b.q.zero_()
    b.q[..., 0] = 8.0
    b.k.zero_()
    for x in keys:
        b.k[x, :, 0] = score / 8   # a bf16 value
    b.v.div_(8)
    b.forward()
    b.check_forward()
    b.backward()
    b.check_backward()
    assert cpt.cpt_kernel_wait_timeouts() == 0


@pytest.mark.parametrize("heads", [(2, 1), (40, 20)])
@pytest.mark.parametrize("second", [-6.0, -2.0, -0.5])
@pytest.mark.parametrize("score", [86.0, 90.0, 94.0])
def test_late_scores_a_little_apart(cpt, cuda_device, score, second, heads):
    """As above with the later of the two a little lower, and a third a little lower still."""
    b = Batch(cpt, 0, 1, [512], *heads, 128, 512, 0, scale=1.0)
    b.q.zero_()
    b.q[..., 0] = 8.0
    b.k.zero_()
    for i, x in enumerate((200, 300, 420)):
        b.k[x, :, 0] = (score + i * second) / 8
    b.forward()
    b.check_forward()
    b.backward()
    b.check_backward()
