"""The bounds-checked build (include/fa_debug.h) over the rotation and the 8-bit cache: silent on valid calls, and with the
same bits as the library's own; with every row extent taken down by one, the last row's accesses are reported."""

import pytest
import torch

from io_aware_exact_04_gb300 import _lib, api
from tests import serving_ref
from tests.test_tree8_gpu import BF16, E4M3, FP16, Made, ints

pytestmark = pytest.mark.gpu
SITES = range(100, 108)


@pytest.fixture
def build(gpu, monkeypatch):
    def use(name):
        lib = _lib.load(name)
        monkeypatch.setattr(api, "_lib_fa", lambda: lib)
        api.device_status(gpu)
        return lib
    yield use
    _lib.load("libfa_debug.so").fa_debug_set_check_slack(0)


def clean(gpu):
    torch.cuda.synchronize(gpu)
    code, detail = api.device_status(gpu)
    assert code == 0, detail


class Tokens:
    def __init__(self, gpu, lens, start, d, page, block, dtype, Hq=6, H=3):
        g = torch.Generator(device=gpu).manual_seed(len(lens) + d)
        self.T, width = sum(lens), -(-max(s + n for s, n in zip(start, lens)) // page)
        self.q, self.k, self.v = (torch.randn((self.T, h, d), generator=g, device=gpu).to(dtype) for h in (Hq, H, H))
        pool = width * len(lens)
        self.table = ints(torch.randperm(pool).view(len(lens), width).tolist(), gpu)
        self.start, self.cu = ints(start, gpu), ints(serving_ref.offsets(lens), gpu)
        self.angles = api.rotary_angles(width * page, d, device=gpu)
        self.wide = [torch.zeros((pool, H, page, d), dtype=dtype, device=gpu) for _ in range(2)]
        self.bytes = [torch.zeros((pool, H, page, d), dtype=torch.uint8, device=gpu) for _ in range(2)]
        self.scales = [torch.ones((pool, H, page // block), device=gpu) for _ in range(2)]

    def eight(self):
        return [x.view(E4M3) for x in self.bytes], dict(k_scale=self.scales[0], v_scale=self.scales[1])

    def rotate(self, wide):
        pages, more = (self.wide, {}) if wide else self.eight()
        return api.rotary_append(self.q, self.k, self.v, *pages, self.table, self.start, self.cu, self.angles, **more)

    def append(self, rows=None, cu=None):
        pages, more = self.eight()
        api.cache_append(self.k, self.v, *pages, self.table, self.start, self.cu if cu is None else cu, rows=rows, **more)

    def all(self, gpu):
        """Every path in turn; what they leave."""
        out = [*self.rotate(True), *self.rotate(False)]
        out += [*api.rotary(self.q, self.k, self.angles, torch.arange(self.T, dtype=torch.int32, device=gpu) % len(self.angles))]
        self.append()
        B = self.cu.numel() - 1
        self.append(rows=torch.arange(B, dtype=torch.int32, device=gpu) % self.T, cu=ints(list(range(B + 1)), gpu))
        clean(gpu)
        return [x.clone() for x in (*out, *self.wide, *self.bytes, *self.scales)]


@pytest.mark.parametrize("dtype", [BF16, FP16])
@pytest.mark.parametrize("d,page,block", [(64, 16, 16), (128, 64, 32), (128, 256, 256), (64, 256, 128)])
@pytest.mark.parametrize("lens,start", [([1, 1, 3, 0, 2], [0, 77, 15, 3, 255]), ([300, 1, 0, 70], [13, 500, 2, 0])])
def test_silent_and_the_same_bits(build, gpu, lens, start, d, page, block, dtype):
    kept = []
    for name in ("libfa_debug.so", "libfa.so"):
        build(name)
        torch.manual_seed(1)
        kept.append(Tokens(gpu, lens, start, d, page, block, dtype).all(gpu))
    assert all(torch.equal(x, y) for x, y in zip(*kept))


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("lens,start", [([1, 1, 3], [0, 77, 15]), ([300, 70], [13, 500])])
def test_rows_past_the_extents_are_reported(build, gpu, lens, start, d):
    lib = build("libfa_debug.so")
    t = Tokens(gpu, lens, start, d, 64, 32, BF16)
    for run in (lambda: t.rotate(True), lambda: t.rotate(False), t.append):
        assert lib.fa_debug_set_check_slack(1) == 0
        run()
        torch.cuda.synchronize(gpu)
        code, detail = api.device_status(gpu)
        assert code == 6 and detail[1] in SITES, detail
        assert lib.fa_debug_set_check_slack(0) == 0
        run()
        clean(gpu)


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("lens,nodes,Hq", [([300, 40], [1, 2], 4), ([9000, 9000], [1, 1], 8), ([300, 700], [40, 33], 8)],
                         ids=["few", "joined", "many"])
def test_results_past_the_extents_are_reported(build, gpu, lens, nodes, Hq, d):
    lib = build("libfa_debug.so")
    m = Made(gpu, lens, nodes, Hq, 2, d, 32, 16, BF16, tail=0)
    m.check()
    assert lib.fa_debug_set_check_slack(1) == 0
    m.call()
    torch.cuda.synchronize(gpu)
    code, detail = api.device_status(gpu)
    assert code == 6 and detail[1] in SITES, detail
    assert lib.fa_debug_set_check_slack(0) == 0
    m.check()
