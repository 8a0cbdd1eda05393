"""What the backward pass of the selective scan reads of the initial state."""
import pytest
import torch

import mamba_ssd_chunked_02_amd as ssd
from block_helpers import offsets, say

pytestmark = pytest.mark.gpu

def test_the_backward_pass_starts_from_the_saved_states():
    """The first of a sequence's saved states is its initial one: the gradients do not read init_state again."""
    say("case: selective scan, initial state of the backward pass")
    lens = [70, 0, 5]
    T, C, N = sum(lens), 16, 16
    g = torch.Generator(device="cuda").manual_seed(1)
    x, dt, dy = (torch.rand(T, C, generator=g, device="cuda") for _ in range(3))
    B, Cm = (torch.rand(T, 1, N, generator=g, device="cuda") for _ in range(2))
    A = -torch.rand(C, N, generator=g, device="cuda")
    init = torch.rand(3, C, N, generator=g, device="cuda")
    kw = dict(cu_seqlens=offsets(lens))
    _, _, states = ssd.selective_scan(x, dt, A, B, Cm, init_state=init, want_states=True, **kw)
    one = ssd.selective_scan_backward(dy, x, dt, A, B, Cm, states, init_state=init, **kw)
    two = ssd.selective_scan_backward(dy, x, dt, A, B, Cm, states, **kw)
    assert all(a is None and b is None or torch.equal(a, b) for a, b in zip(one, two))
