"""The status word is shared by everything on a device: a recorded check (a bad page id, say: documented, the call
carries on) does not hide a wait that ran out.
"""

import pytest
import torch

from io_aware_exact_04_gb300 import _lib, api
from test_serving_gpu import Cache, ints, rows_like

pytestmark = pytest.mark.gpu

TIMEOUT = 5


@pytest.mark.parametrize("d", [64, 128])
def test_a_timeout_replaces_a_recorded_check(gpu, monkeypatch, d):
    """In the build that leaves out a copy in every CTA: a bad page id, then the wait that runs out."""
    lib = _lib.load("libfa_withhold.so")
    monkeypatch.setattr(api, "_lib_fa", lambda: lib)
    api.device_status(gpu)
    c = Cache([4000], 1, 64, d, torch.bfloat16, gpu)
    table = c.table.clone()
    table[0, 0] = 1 << 20
    q, k, v = rows_like("plain", 1, 4, 1, d, torch.bfloat16, gpu)
    api.forward_tree(q, k, v, c.kv[0], c.kv[1], table, c.lens, ints([0, 1], gpu))
    torch.cuda.synchronize(gpu)
    code, detail = api.device_status(gpu)
    assert code == TIMEOUT and detail[0] == TIMEOUT and 60 <= detail[1] <= 72, detail
    assert api.device_status(gpu)[0] == 0
