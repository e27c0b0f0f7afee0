"""What a captured decode of a short table leaves behind."""
import gc

import pytest
import torch

import quantized_paged_attention_gb300 as qpa
from _gpu import bf16_tensor, dev
from test_gpu_nvfp4 import Case, done, f32, t32

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("on_stream", [False, True])
def test_a_captured_first_call_keeps_nothing_of_its_graph(on_stream):
    """The first short decode of a process under capture: once the graph and its output are gone, so is all memory that
    the call took, and a call outside gives the same."""
    c = Case([100, 7], 2, 4, 128, 16)
    q, table, lens = bf16_tensor(c.q, dev()), t32(c.table), t32(c.lens)
    cache, ks, vs = torch.from_numpy(c.cache).to(dev()), f32(c.gs[0]), f32(c.gs[1])
    ws = qpa.alloc_workspace(qpa.pa_decode_nvfp4_workspace_size(qpa.nvfp4_desc(q, cache, table, 4)), dev())
    want = c.run(workspace=ws)
    done()
    qpa._DECODE4_UNTOUCHED.clear()
    gc.collect()
    torch.cuda.empty_cache()
    before = torch.cuda.memory_allocated(), torch.cuda.memory_reserved()
    g, side = torch.cuda.CUDAGraph(), torch.cuda.Stream()
    with torch.cuda.graph(g, stream=side):
        out = qpa.pa_decode_nvfp4(q, cache, table, lens, ks, vs, 4, stream=side if on_stream else None)
    g.replay()
    torch.cuda.synchronize()
    assert torch.equal(out, want)
    del out, g
    gc.collect()
    torch.cuda.synchronize()
    torch.cuda.empty_cache()
    assert (torch.cuda.memory_allocated(), torch.cuda.memory_reserved()) == before
    outs = [c.run(), c.run()]
    done()
    assert all(torch.equal(o, want) for o in outs)
