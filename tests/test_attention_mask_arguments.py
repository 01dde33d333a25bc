"""The window and the sinks that the binding hands to the library."""
import pytest
import torch


class Calls:
    """Stands in for the library: takes the arguments down."""

    def __init__(self):
        self.seen = []

    def cpt_attention(self, *a):
        self.seen.append(a[11:13])
        return 0

    def cpt_attention_backward(self, *a):
        self.seen.append(a[15:17])
        return 0


@pytest.mark.parametrize("window,sinks,want", [
    (4, 2, (4, 2)), (0, 0, (0, 0)), (2 ** 63 - 1, 2 ** 31 - 1, (2 ** 63 - 1, 2 ** 31 - 1)),
    (2 ** 63, 2 ** 31, (2 ** 63 - 1, 2 ** 31 - 1)), (2 ** 64, 2 ** 32, (2 ** 63 - 1, 2 ** 31 - 1)),
    (2 ** 64 + 5, 2 ** 32 + 5, (2 ** 63 - 1, 2 ** 31 - 1)), (-1, -1, (-1, -1)), (-2 ** 64, -2 ** 32, (-1, -1))])
def test_values_beyond_the_types_are_not_cut(cpt, monkeypatch, window, sinks, want):
    fake = Calls()
    monkeypatch.setattr(cpt, "_lib", fake)
    plan = cpt.Plan(0, None, 0, 2, 1, 16, 16)
    bf = torch.bfloat16
    q, k, lse = torch.zeros(16, 4, 8, dtype=bf), torch.zeros(16, 2, 8, dtype=bf), torch.zeros(4, 16)
    w = [torch.zeros(16, 2, 8, dtype=bf) for _ in range(2)]
    cpt.cpt_attention(plan, q, k, k, q, lse, 1.0, window, sinks, stream=0)
    cpt.cpt_attention_backward(plan, q, k, k, q, lse, q, q, w, w, 1.0, window, sinks,
                               workspace=torch.zeros(256, dtype=torch.uint8), stream=0)
    assert fake.seen == [want, want]
