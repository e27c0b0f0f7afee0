"""How the decode cuts its work: the pieces that it leaves in the workspace against the
restatement of the ranges."""
import numpy as np
import pytest
import torch

import quantized_paged_attention_gb300 as qpa
from _gpu import dev
from test_gpu_nvfp4 import done, f32, t32
from test_nvfp4_schedule import TILE, _ranges

pytestmark = pytest.mark.gpu
MAX_CTAS = 160                          # the workspace has two slots of 16 rows for each, then their {m, l}, then a record per CTA
BEGIN = {64: 8, 128: 5}


def ctas_of(units):
    return min(units, torch.cuda.get_device_properties(dev()).multi_processor_count, MAX_CTAS)


@pytest.mark.parametrize("seed", range(40))
def test_pieces_left_in_the_workspace(seed):
    """Keys of zeros: every logit is 0, a token weighs 2^8, and a piece's sum of weights counts its tokens (exact below 2^16
    tokens). Each slot that the restated ranges give a piece holds that piece's tokens; each CTA's record says how many
    pieces the item that begins there and goes on has."""
    r = np.random.default_rng(seed)
    D, G = [(128, 4), (64, 8), (128, 16), (64, 33)][seed % 4]
    Hk, bs, RB = int(r.choice([1, 2, 5])), 64, -(-G // 16)
    top = int(r.choice([700, 5000, 60000]))
    lens = r.choice([0, 1, 128, 129], 40)
    long = r.random(40) < 0.6
    lens[long] = r.integers(1, top, int(long.sum()))
    lens = lens[:int(r.integers(1, 41))]
    lens[0] = top
    B, maxb = len(lens), -(-top // bs)
    cache = torch.zeros(*qpa.nvfp4_cache_shape(1, Hk, bs, D), dtype=torch.uint8, device=dev())
    table = torch.zeros(B, maxb, dtype=torch.int32, device=dev())
    q = torch.ones(B, Hk * G, D, dtype=torch.bfloat16, device=dev())
    ws = torch.full((qpa.pa_decode_nvfp4_workspace_size(qpa.nvfp4_desc(q, cache, table, G)),), 0xFF, dtype=torch.uint8, device=dev())
    qpa.pa_decode_nvfp4(q, cache, table, t32(lens), f32(1.0), f32(1.0), G, workspace=ws)
    done()
    ctas = ctas_of(-(-maxb * bs // TILE) * B * Hk * RB)
    slots = 2 * MAX_CTAS * 16
    raw = ws.cpu().numpy()
    ml = raw[slots * D * 4:slots * (D * 4 + 8)].view(np.float32).reshape(2 * MAX_CTAS, 16, 2)
    meta = raw[slots * (D * 4 + 8):][:MAX_CTAS * 16].view(np.int32).reshape(MAX_CTAS, 4)
    tiles, ranges, told = _ranges(lens.tolist(), Hk * RB, ctas, BEGIN[D], False)
    pieces = 0
    for cta, items in enumerate(ranges):
        want = (0, 0, 0)
        for s, vh, t, te in items:
            if t == 0 and te < tiles[s]:
                want = (told[s, vh], s, vh)
            if t > 0 or te < tiles[s]:
                rows = min(16, G - 16 * (vh % RB))
                got = ml[2 * cta + (t == 0), :rows]
                assert np.all(got[:, 0] == -8) and np.all(got[:, 1] == 256 * (min(te * TILE, lens[s]) - t * TILE)), (cta, s, vh, t, te)
                pieces += 1
        assert tuple(meta[cta, :3]) == want or want[0] == 0 == meta[cta, 0], (cta, want, meta[cta])
    assert pieces == sum(told.values())
