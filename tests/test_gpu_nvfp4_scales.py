"""pa_decode_nvfp4 with tensor scales at the ends of float32."""
import numpy as np
import pytest
import torch

import oracle
import quantized_paged_attention_gb300 as qpa
import synth
from _gpu import bf16_tensor, dev
from test_gpu_nvfp4 import done, f32, rand_cache, rand_table, t32

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("D,G,bs,lens,cols", [(128, 8, 16, [4000, 300, 1], 1), (64, 16, 32, [9000], 1), (64, 3, 128, [500, 20], 0)])
@pytest.mark.parametrize("g", [1e-36, -3e-35, 2.0 ** -132, 1e33])
def test_value_scales(D, G, bs, lens, cols, g):
    """Results keep bf16's bits however small v_scale is. Tolerance: as the other decodes, and 2^-133 (bf16's smallest step,
    half of it for the rounding of a result below 2^-126, less for float32's before). The last case has a table of 512 tokens."""
    r = synth.rng(D + G)
    table, NB = rand_table(r, lens, bs, cols=cols)
    cache, lens = rand_cache(r, NB, 2, bs, D, smax=127), np.array(lens)
    q = synth.round_to_bf16_bits(0.2 * r.standard_normal((len(lens), 2 * G, D)))
    want, bound, total, slack = oracle.pa_decode_nvfp4(q, cache, table, lens, .02, g, G)
    out = qpa.pa_decode_nvfp4(bf16_tensor(q, dev()), torch.from_numpy(cache).to(dev()), t32(table), t32(lens), f32(.02), f32(g), G)
    done()
    tol = 2.0 ** -8 * np.abs(want) + bound * (2 * 2.0 ** -11 + 2 * np.expm1(slack)[..., None] + 2.0 ** -18)
    tol += 2.0 ** -33 * (total + lens[:, None, None] * np.abs(want)) + 2.0 ** -133
    err = np.abs(out.float().cpu().numpy().astype(np.float64) - want)
    assert np.all(err <= tol), (err / tol).max()
