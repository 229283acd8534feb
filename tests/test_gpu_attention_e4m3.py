"""The two kernels of dspark_tree_attention over an 8-bit cache: eight query rows of a
kv head at once, or up to 128.  Which of them does a call is the library's choice; here
the second is asked for by scales that do not lie on 16 bytes, which the first does not
take, so that no choice of the library takes it out of its tests."""

import math

import pytest
import torch

import window_oracle as wo
from gpu_helpers import require_gpu
from test_gpu_attention import Problem

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def api():
    require_gpu()
    from confidence_scheduled_speculative_gb300 import api
    return api


def _off_16_bytes(t):
    """The same tensor 4 bytes past a 16-byte boundary."""
    flat = torch.empty(t.numel() + 4, device=t.device, dtype=t.dtype)
    moved = flat[1:1 + t.numel()].view(t.shape)
    assert moved.data_ptr() % 16 == 4
    return moved.copy_(t)


class Wide(Problem):
    """A problem for the kernel of 128 rows."""

    def run(self, api, lse=True):
        c = self.cache
        if c.k_scale.data_ptr() % 16 == 0:
            c.k_scale, c.v_scale = _off_16_bytes(c.k_scale), _off_16_bytes(c.v_scale)
        return super().run(api, lse)


# ------------------------------------------------------------ which one

def _wide_did(api, shape):
    """Whether the bits of a call are those of the kernel of 128 rows."""
    a = Problem(600, kind="e4m3", **shape).run(api)
    b = Wide(600, kind="e4m3", **shape).run(api)
    a.check()
    b.check()
    return torch.equal(a.out, b.out) and torch.equal(a.lse, b.lse)


G4, G8 = dict(hq=8, hkv=2, D=128, page=64), dict(hq=16, hkv=2, D=128, page=64)


@pytest.mark.parametrize("wide,shape", [
    # long windows of two requests among slots without a row, one tree over a long prefix
    # beside single tokens, whatever the rows of the call have room for
    (True, dict(prefix=[3000, 2500] + [900] * 62, win=[32, 32] + [0] * 62, pad=0, **G8)),
    (True, dict(prefix=[40000] + [70] * 63, win=[32] + [1] * 63, pad=33, **G4)),
    (True, dict(prefix=[3000] * 8 + [9] * 24, win=[8] * 8 + [0] * 24, pad=0, **G4)),
    (True, dict(prefix=[3000] * 4, win=[32] * 4, pad=64, **G4)),
    # single tokens, beside slots without one and beside a long window over nothing much
    (False, dict(prefix=[3000] * 20, win=[1] * 20, pad=0, **G4)),
    (False, dict(prefix=[3000] * 20, win=[1] * 20, pad=400, **G4)),
    (False, dict(prefix=[3000] * 9 + [50] * 80, win=[1] * 9 + [0] * 80, pad=3, **G8)),
    (False, dict(prefix=[30000, 0], win=[1, 32], pad=0, **G4)),
])
def test_the_work_decides(api, wide, shape):
    """Passes over the long prefixes decide, not rows over requests."""
    assert _wide_did(api, shape) == wide
