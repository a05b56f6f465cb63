"""How far a NaN or an infinity in a token reaches that its reader does not see."""

import pytest
import torch

import serving_ref as ref
from io_aware_exact_04_gb300 import api
from test_serving_gpu import Cache, ints, masks_of, ok, rows_like

pytestmark = pytest.mark.gpu


def reached(got, clean):
    """[T, Hq]: whose rows differ from the clean call's."""
    return (got.view(torch.int16) != clean.view(torch.int16)).any(-1)


@pytest.mark.parametrize("bad", [float("nan"), float("inf")])
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("G", [1, 2, 3, 5, 7, 16, 128])
def test_prompt_values(gpu, G, d, bad):
    """V of one token: its own and later tokens of its head see it; earlier ones may be reached only where less
    than 128 + 128 // G before it, other heads and other sequences never."""
    n, Hkv, reach = 520, 2, 128 + 128 // G
    q, k, v = rows_like("plain", 2 * n, G * Hkv, Hkv, d, torch.bfloat16, gpu, seed=G)
    cu = ints([0, n, 2 * n], gpu)
    clean, lse = api.forward_prompt(q, k, v, cu)
    for j in (0, 63, 128, 167, 255, 256, 300, 383, 419, 511, 519):
        x = v.clone()
        x[j, 1] = bad
        got, glse = api.forward_prompt(q, k, x, cu)
        ok(gpu)
        hit = reached(got, clean)
        assert not hit[:, :G].any() and not hit[n:].any(), "another head or sequence"
        assert torch.equal(glse, lse)
        first = j if not hit[:j].any() else int(hit[:j].any(1).nonzero()[0])
        assert j - first < reach, (j, first)
        assert not torch.isfinite(got[j:n, G:].float()).any()


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("G", [1, 3, 16])
def test_prompt_keys(gpu, G, d):
    """K of one token never reaches the tokens before it."""
    n = 520
    q, k, v = rows_like("plain", n, G, 1, d, torch.float16, gpu, seed=G)
    cu = ints([0, n], gpu)
    clean, lse = api.forward_prompt(q, k, v, cu)
    for j in (1, 127, 300, 511):
        x = k.clone()
        x[j] = float("nan")
        got, glse = api.forward_prompt(q, x, v, cu)
        ok(gpu)
        assert torch.equal(got[:j], clean[:j]) and torch.equal(glse[:, :j], lse[:, :j])
        assert torch.isnan(got[j:].float()).all() and torch.isnan(glse[:, j:]).all()


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("G", [1, 4])
def test_tree_nodes(gpu, G, d):
    """A node's K reaches the nodes that see it and no others; its V its own sequence and head only."""
    lens, nodes, Hkv = [200, 0, 64], [9, 40, 130], 2
    T = sum(nodes)
    q, k, v = rows_like("plain", T, G * Hkv, Hkv, d, torch.bfloat16, gpu, seed=G)
    c = Cache(lens, Hkv, 32, d, torch.bfloat16, gpu)
    words, bits, _ = masks_of("tree", nodes)
    mask = torch.cat([ref.pack_bits(s, words) for s in bits]).to(gpu)
    cu, at = ints(ref.offsets(nodes), gpu), ref.offsets(nodes)
    clean, lse = api.forward_tree(q, k, v, c.kv[0], c.kv[1], c.table, c.lens, cu, mask=mask)
    for b, n in enumerate(nodes):
        for i in (0, n // 2, n - 1):
            x = k.clone()
            x[at[b] + i, 0] = float("nan")
            got, glse = api.forward_tree(q, x, v, c.kv[0], c.kv[1], c.table, c.lens, cu, mask=mask)
            ok(gpu)
            seen = torch.zeros(T, dtype=torch.bool)
            seen[at[b]:at[b + 1]] = bits[b][:, i]
            assert torch.equal(torch.isnan(glse[:G]).all(0).cpu(), seen) and torch.equal(glse[G:], lse[G:])
            assert torch.equal(reached(got, clean)[:, :G].all(1).cpu(), seen) and not reached(got, clean)[:, G:].any()
            x = v.clone()
            x[at[b] + i, 0] = float("inf")
            got, glse = api.forward_tree(q, k, x, c.kv[0], c.kv[1], c.table, c.lens, cu, mask=mask)
            ok(gpu)
            hit = reached(got, clean)
            assert torch.equal(glse, lse) and not hit[:, G:].any()
            assert not hit[:at[b]].any() and not hit[at[b + 1]:].any() and bool(hit[:, :G][seen.to(gpu)].all())
