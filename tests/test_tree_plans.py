"""Host-only: what plans of tree attention ask for stays in proportion to the work."""
import random

import pytest

import gemm_conv_chain_amd as fc

pytestmark = pytest.mark.cpu


def test_no_workspace_for_parts_that_nothing_is_left_for():
    """150 small trees over some hundred keys have a few stages of 64 each: 1024 splits are
    no more of them, nor a workspace of gigabytes."""
    few = fc.attn_plan(1800, 150, 4, 2, 64, 16, 7, 12, 102, variant="tile", splits=3, tree=True)
    many = fc.attn_plan(1800, 150, 4, 2, 64, 16, 7, 12, 102, variant="tile", splits=1024, tree=True)
    assert many["splits"] <= 4 and few["workspace"] <= many["workspace"] < 64 << 20


@pytest.mark.parametrize("seed", range(200))
def test_workspace_is_bounded_by_the_stages(seed):
    rng = random.Random(seed)
    d, page, hkv, G = rng.choice([64, 128, 192, 256]), rng.choice([16, 64, 256]), rng.choice([1, 2, 8]), rng.choice([1, 4, 7])
    batch, max_q, max_kv = rng.choice([1, 3, 40, 1000]), rng.choice([1, 8, 60, 500]), rng.choice([1, 20, 300, 5000])
    stride = -(-max_kv // page)
    window = rng.choice([0, 0, 100])
    stages = batch * (-(-max_kv // 16) + 1) * 16 // (64 if d <= 192 else 32) + 2 * batch
    rows = 128 if d <= 128 else 256
    tiles = -(-max_q * G // rows)
    for splits in (0, 1, 2, 7, 100, 1024):
        p = fc.attn_plan(batch * max_q, batch, hkv * G, hkv, d, page, stride, max_q, max_kv, variant="tile", splits=splits,
                         window=window, tree=True)
        assert p["variant"] == "tile" and p["splits"] <= max(splits, 1) or splits == 0
        slots = min(splits * batch if splits else stages, stages) + batch
        assert p["workspace"] <= slots * tiles * rows * hkv * (d + 4) * 4 + 8 * batch
        assert splits != 1 or p["workspace"] == 0
