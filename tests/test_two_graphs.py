"""Graphs of different sizes live side by side in a process (a drafting model
and the model that judges its tokens): binding one leaves the others able to
run."""
import numpy as np
import pytest
import torch

from task_graph_runtime_gb300 import mpk, synth

from gpu_util import dev_kv, dev_weights

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("mode", [mpk.MODE_MEGAKERNEL, mpk.MODE_KPO])
def test_a_graph_bound_later_with_less_shared_memory(mode):
    small = synth.ModelShape(1, 64, 2, 1, 32, 64, 100)
    big = synth.ModelShape(1, 1024, 8, 2, 128, 4096, 1000)
    out = []
    graphs = []
    for shape, batch in ((big, 8), (small, 2)):
        wl = synth.Workload("w", shape, batch, (17,) * batch, 16, 4)
        g = mpk.Graph(shape, batch, page_size=16,
                      max_pages_per_seq=wl.max_pages_per_seq)
        g.bind(dev_weights(synth.model_weights(shape, 1), shape))
        g.set_mode(mode)
        kv = synth.kv_inputs(wl, 1)
        tok = torch.from_numpy(synth.tokens(wl, 1)).cuda()
        graphs.append((g, kv, tok, batch, shape.vocab))
        if shape is big:        # alone in the process so far
            out.append(_step(*graphs[0]))
    for i in (0, 1, 0):
        got = _step(*graphs[i])
        if i == 0:
            assert np.array_equal(got, out[0])
    for g, *_ in graphs:
        g.close()


def _step(g, kv, tok, batch, vocab):
    lg = torch.empty(batch, vocab, device="cuda")
    nt = torch.empty(batch, dtype=torch.int32, device="cuda")
    g.decode_step(tok, dev_kv(kv), lg, nt)
    torch.cuda.synchronize()
    assert g.status() == mpk.MPK_OK
    return lg.cpu().numpy()
